/*
 * lstm_ops.h -- the part of liblstmstack.so's C ABI for state-space sequence
 * layers and for reading a model's answers off its logits:
 *  - lstm_causal_conv, lstm_causal_conv_step: the short causal depthwise
 *    convolution over prompts, and over the next token of each sequence;
 *  - lstm_selective_scan, lstm_selective_scan_step: the selective state space
 *    recurrence over prompts, and over the next token of each sequence;
 *  - lstm_residual_rms_norm: a residual's addition and the root-mean-square
 *    norm of the sum, in the input's type or in 8 bits with scales;
 *  - lstm_token_logprobs: log probabilities of given tokens, the entropy and
 *    the top alternatives of each row of logits.
 *
 * The conventions of lstm_stack.h hold (device pointers, streams, return
 * codes, lstm_stack_last_error), with these differences:
 *  - Activations have one of the LSTM_F32, LSTM_BF16 and LSTM_F16 types, the
 *    same for all of one call's; weights and the scan's states are fp32.
 *    Everything is computed in fp32 and rounded once, when it is stored.
 *  - A matrix [rows][cols] has consecutive columns and a row stride counted
 *    in elements, at least cols (so it may be a slice of wider rows).  Any
 *    element-aligned address and any stride are taken; rows that start on
 *    16-byte boundaries move faster.
 *  - Weights, biases and states are densely packed, at any element-aligned
 *    address.
 *  - The calls allocate nothing, keep nothing between calls, wait for nothing
 *    and can be captured into a CUDA graph (after one call on the device
 *    outside a capture).  Outputs must not overlap inputs unless stated.
 *
 * Sequences.  `tokens` rows hold `sequences` sequences one after the other
 * without padding: sequence s is the rows offsets[s] .. offsets[s+1]-1
 * (device int32 [sequences + 1], not decreasing, from 0 to tokens; bounds
 * outside 0..tokens are clamped), or with offsets NULL every sequence has
 * tokens / sequences rows (tokens must be a multiple of sequences).  Lengths
 * may be zero.  A call has at most LSTM_MAX_SEQUENCES sequences and 2^31 - 256
 * tokens (more: LSTM_E_OVERFLOW).
 *
 * States.  A pool of `state_slots` states holds what a sequence needs to go
 * on with its next tokens.  Sequence s has slot slots[s] (device int32
 * [sequences]; NULL: slot s); a slot outside 0..state_slots-1 means no state:
 * the sequence starts from zeros and stores nothing.  No two sequences of a
 * call may share a slot.  A prompt starts from its slot's state where
 * resume[s] is non-zero (device int32 [sequences]; NULL: none does), else
 * from zeros, and leaves its last state in the slot; a step always goes on
 * from its slot's state.
 */
#ifndef LSTM_OPS_H
#define LSTM_OPS_H

#include "lstm_stack.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of activations. */
enum {
    LSTM_F32 = 0,
    LSTM_BF16 = 1,
    LSTM_F16 = 2,
    LSTM_E4M3 = 3 /* 8 bits, 4 of exponent; lstm_residual_rms_norm's output only */
};

#define LSTM_MAX_SEQUENCES (1 << 30)
#define LSTM_CONV_MAX_WIDTH 4
#define LSTM_SCAN_MAX_STATES 128
#define LSTM_TOP_MAX 32

/* y[t][d] = act(bias[d] + sum_k w[d][k] * x[t - (width-1) + k][d]), each
 * sequence for itself; before a sequence's first row stand its state's rows,
 * or zeros.  act(v) = v / (1 + e^-v) with silu != 0, else v.
 *   x, y  : device [tokens][channels], row strides x_stride, y_stride
 *   w     : device [channels][width] fp32, 2 <= width <= LSTM_CONV_MAX_WIDTH
 *   bias  : device [channels] fp32, or NULL
 *   state : device [state_slots][width-1][channels] of x's type, the last
 *           width-1 inputs, oldest first; NULL: no states (state_slots,
 *           slots and resume are then not read)
 * Errors: LSTM_E_INVALID (null, sizes, type, stride, device), LSTM_E_LENGTH
 * (offsets NULL and tokens no multiple of sequences), LSTM_E_OVERFLOW,
 * LSTM_E_DEVICE, LSTM_E_CUDA. */
int lstm_causal_conv(const void *x, long long x_stride, int dtype, int tokens, int channels,
                     int width, const float *w, const float *bias, int silu, int sequences,
                     const int *offsets, void *state, int state_slots, const int *slots,
                     const int *resume, void *y, long long y_stride, void *stream);

/* The next token of every sequence: row s of x and y (device
 * [sequences][channels]) is sequence s's, and its state moves on by one
 * input.  Arguments and errors as lstm_causal_conv; state is required. */
int lstm_causal_conv_step(const void *x, long long x_stride, int dtype, int sequences,
                          int channels, int width, const float *w, const float *bias, int silu,
                          void *state, int state_slots, const int *slots, void *y,
                          long long y_stride, void *stream);

/* The selective scan, each sequence for itself and each channel d with
 * `states` states h[n]:
 *   s      = dt[t][d] + dt_bias[d], and log(1 + e^s) of it with softplus != 0
 *   h[n]   = e^(s * a[d][n]) * h[n] + s * u[t][d] * b[t][g][n]
 *   v      = sum_n h[n] * c[t][g][n] + skip[d] * u[t][d]
 *   y[t][d] = v * z / (1 + e^-z), z = z[t][d]
 * where g = d / (channels / groups).
 *   u, dt, z, y : device [tokens][channels]; z NULL: no gate, y = v
 *   a           : device [channels][states] fp32 (negative: a decay),
 *                 1 <= states <= LSTM_SCAN_MAX_STATES
 *   b, c        : device [tokens][groups][states] (a row's groups * states
 *                 values consecutive); groups divides channels
 *                 (channels and groups * states: at most 2^30, else
 *                 LSTM_E_OVERFLOW)
 *   skip, dt_bias : device [channels] fp32, or NULL: nothing is added
 *   state       : device [state_slots][channels][states] fp32, the h; NULL:
 *                 no states (state_slots, slots and resume are then not read)
 *   workspace   : device, 16-byte aligned, workspace_bytes long and at least
 *                 lstm_selective_scan_workspace(tokens, channels, states,
 *                 groups, sequences, offsets == NULL) bytes (0: may be NULL);
 *                 its contents need not be kept between calls, but two calls
 *                 that may run at the same time need one each
 * Errors as lstm_causal_conv, LSTM_E_LENGTH for a workspace that is too short. */
size_t lstm_selective_scan_workspace(int tokens, int channels, int states, int groups,
                                     int sequences, int equal_lengths);
int lstm_selective_scan(const void *u, long long u_stride, const void *dt, long long dt_stride,
                        const float *a, const void *b, long long b_stride, const void *c,
                        long long c_stride, const float *skip, const void *z, long long z_stride,
                        const float *dt_bias, int softplus, int dtype, int tokens, int channels,
                        int states, int groups, int sequences, const int *offsets, float *state,
                        int state_slots, const int *slots, const int *resume, void *y,
                        long long y_stride, void *workspace, size_t workspace_bytes, void *stream);

/* The next token of every sequence: row s of u, dt, b, c, z and y is sequence
 * s's, and its state moves on by one token.  Arguments and errors as
 * lstm_selective_scan; state is required.  A copy of states that does not
 * arrive within two seconds sets the library's fault word (lstm_fault_status);
 * the call's outputs and states are then unspecified. */
int lstm_selective_scan_step(const void *u, long long u_stride, const void *dt,
                             long long dt_stride, const float *a, const void *b,
                             long long b_stride, const void *c, long long c_stride,
                             const float *skip, const void *z, long long z_stride,
                             const float *dt_bias, int softplus, int dtype, int sequences,
                             int channels, int states, int groups, float *state, int state_slots,
                             const int *slots, void *y, long long y_stride, void *stream);

/* v = x + residual (x alone with residual NULL) and its norm
 *   n[r][c] = v[r][c] / sqrt(mean_c v[r][c]^2 + eps) * weight[c].
 * residual_out receives v rounded to x's type (residual_out may be residual);
 * the norm is taken of the unrounded v.
 *   x, residual, residual_out : device [rows][cols] of type dtype; residual
 *            and residual_out are both given or both NULL
 *   weight : device [cols] fp32
 *   y      : device [rows][cols] of type y_dtype: dtype, or LSTM_E4M3
 *   scales : with LSTM_E4M3, device [rows][ceil(cols / group)] fp32, group
 *            one of 32, 64 and 128, or 0 for one scale a row; else not read.
 *            A scale is the largest |n| of its columns / 448, at least
 *            2^-126, and 1 where all are 0; y = n / scale rounded to nearest
 *            even (both quotients as fp32 division rounds them), so y * scale
 *            stands for n.
 * A row that holds infinities or NaN gives NaN where IEEE arithmetic does.
 * Squares are summed in fp32: a row whose sum of squares is above 3.4e38 (values
 * of 1e19 and more) has a norm of 0, as one with an infinity has, and squares
 * below 1e-45 add nothing to eps.
 * 1 <= cols <= 32768.  Errors: LSTM_E_INVALID, LSTM_E_OVERFLOW,
 * LSTM_E_DEVICE, LSTM_E_CUDA. */
int lstm_residual_rms_norm(const void *x, long long x_stride, const void *residual,
                           long long residual_stride, int dtype, const float *weight, float eps,
                           int rows, int cols, void *residual_out, long long residual_out_stride,
                           void *y, long long y_stride, int y_dtype, float *scales, int group,
                           void *stream);

/* For each row of logits (device [rows][vocab], row stride `stride`), with
 * l = log softmax of the row:
 *   logp[r]    = l[tokens[r]]         tokens: device int64 [rows]; a negative
 *                token asks for nothing and gives 0, one >= vocab gives NaN
 *   entropy[r] = -sum_v e^l[v] l[v]   (terms with e^l = 0 are 0)
 *   top_ids[r][0..top-1], top_logp[r][..] : the `top` largest logits' indices
 *                (int64) and their l, largest first, equal logits in the order
 *                of their indices; 0 <= top <= min(vocab, LSTM_TOP_MAX)
 * logp and tokens may both be NULL, entropy may be NULL, and with top 0
 * top_logp and top_ids are not written.  Logits of -infinity (masked) have
 * probability 0; a row of nothing else has l = -infinity everywhere and
 * entropy 0.  A row with a NaN or +infinity has l and entropy NaN, and NaN
 * counts as the largest logit.  Errors: LSTM_E_INVALID, LSTM_E_OVERFLOW,
 * LSTM_E_DEVICE, LSTM_E_CUDA. */
int lstm_token_logprobs(const void *logits, long long stride, int dtype, int rows, int vocab,
                        const long long *tokens, float *logp, float *entropy, int top,
                        float *top_logp, long long *top_ids, void *stream);

/* Failure-injection hook, as lstm_test_recurrence_timeout: with withhold != 0
 * lstm_selective_scan_step asks for no copies of states where it works on whole
 * tiles of them, so that the waits for them run out. */
int lstm_test_scan_step_timeout(int withhold, unsigned int wait_limit_us, int device);

#ifdef __cplusplus
}
#endif

#endif /* LSTM_OPS_H */
