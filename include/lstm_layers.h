/*
 * lstm_layers.h -- the part of liblstmstack.so's C ABI for layers whose state
 * is a matrix per head, and for the dense products around them:
 *  - lstm_linear_attention, lstm_linear_attention_step: linear attention with a
 *    decay for each head over prompts, and over the next token of each sequence;
 *  - lstm_dense: a matrix product with bias, activation and residual.
 *
 * The conventions of lstm_ops.h hold: its element types, matrices with row
 * strides, packed sequences, pools of states, and its return codes.
 */
#ifndef LSTM_LAYERS_H
#define LSTM_LAYERS_H

#include "lstm_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LSTM_ATTENTION_MAX_KEYS 128
#define LSTM_ATTENTION_MAX_VALUES 256
#define LSTM_ATTENTION_MAX_HEADS 32768

/* Linear attention, each sequence for itself and each head h with a state S of
 * `keys` x `values` numbers:
 *   S          = e^(log_decay[t][h]) * S + k[t] v[t]^T
 *   y[t][h][c] = scale * sum_n q[t][n] * S[n][c]
 * with q, k and v of head h's group.
 *   q, k : device [tokens][q_heads or k_heads][keys]; consecutive keys, the
 *          heads of a token *_head_stride elements apart (not read for one
 *          head) and the tokens *_stride, each at least keys (so a token's
 *          heads may lie side by side, or all tokens of a head)
 *   v    : device [tokens][v_heads][values], as q and k
 *          q_heads, k_heads and v_heads divide heads; head h has the head
 *          h / (heads / q_heads) of q, and so on
 *   log_decay : device fp32, decay_stride 0: [heads], the same for every
 *          token; else [tokens][heads] with that row stride (at least heads).
 *          A value of -infinity forgets the state; values are below 88, and so
 *          is every sum of a sequence's consecutive values (e^88 is beyond fp32:
 *          y and states may be NaN, even where zeros hide the growth)
 *   y    : device [tokens][heads][values], the heads of a token consecutive
 *          and the tokens y_stride apart (at least heads * values)
 *   state : device [state_slots][heads][keys][values] fp32, or NULL: no
 *          states (state_slots, slots and resume are then not read)
 *   workspace : device, 16-byte aligned, workspace_bytes long and at least
 *          lstm_linear_attention_workspace(...) bytes of the same sizes (0:
 *          may be NULL); its contents need not be kept between calls, but two
 *          calls that may run at the same time need one each
 * 1 <= keys <= LSTM_ATTENTION_MAX_KEYS, 1 <= values <=
 * LSTM_ATTENTION_MAX_VALUES, 1 <= heads <= LSTM_ATTENTION_MAX_HEADS.
 * States are fp32.  Products are the tensor cores', whose fp32 sums are cut off
 * below their last bit, of numbers as parts of bf16.  What a token adds to a
 * state goes as three parts, 24 bits (its decay's exponential is good to 2^-22).
 * With 16-bit types the products that make y take the state and the products of
 * queries and keys rounded to 16 bits (two parts of bf16), and LSTM_F16 leaves 2^-16
 * of a product out at most.
 * With LSTM_F32 every factor goes as three parts: a product loses 2^-24 of itself
 * at most, and what of its factors lies below 2^-133.
 * An infinity or a NaN, or a product beyond fp32, makes what depends on it, itself
 * or through a state, infinite (of either sign) or NaN; tokens before it, other heads
 * and sequences are as without.
 * Few sequences and heads are cut into spans that run side by side (whence the
 * workspace): a state's sums are then made in another order, which sizes alone
 * decide, so that the same call gives the same bits.
 * A wait inside the kernel that does not end within some eight seconds sets the
 * library's fault word (lstm_fault_status); outputs and states are then
 * unspecified.
 * Errors: LSTM_E_INVALID (null, sizes, type, stride, device), LSTM_E_LENGTH
 * (offsets NULL and tokens no multiple of sequences; a workspace that is too
 * short), LSTM_E_OVERFLOW, LSTM_E_DEVICE, LSTM_E_CUDA. */
size_t lstm_linear_attention_workspace(int tokens, int heads, int keys, int values, int sequences,
                                       int equal_lengths);
int lstm_linear_attention(const void *q, long long q_stride, long long q_head_stride, int q_heads,
                          const void *k, long long k_stride, long long k_head_stride, int k_heads,
                          const void *v, long long v_stride, long long v_head_stride, int v_heads,
                          const float *log_decay, long long decay_stride, float scale, int dtype,
                          int tokens, int heads, int keys, int values, int sequences,
                          const int *offsets, float *state, int state_slots, const int *slots,
                          const int *resume, void *y, long long y_stride, void *workspace,
                          size_t workspace_bytes, void *stream);

/* The next token of every sequence: row s of q, k, v, log_decay and y is
 * sequence s's, and its state moves on by one token, all in fp32.  Arguments
 * and errors as lstm_linear_attention; state is required. */
int lstm_linear_attention_step(const void *q, long long q_stride, long long q_head_stride,
                               int q_heads, const void *k, long long k_stride,
                               long long k_head_stride, int k_heads, const void *v,
                               long long v_stride, long long v_head_stride, int v_heads,
                               const float *log_decay, long long decay_stride, float scale,
                               int dtype, int sequences, int heads, int keys, int values,
                               float *state, int state_slots, const int *slots, void *y,
                               long long y_stride, void *stream);

/* Activations of lstm_dense. */
enum {
    LSTM_ACT_NONE = 0,
    LSTM_ACT_RELU = 1,      /* max(v, 0) */
    LSTM_ACT_GELU = 2,      /* v (1 + erf(v / sqrt 2)) / 2 */
    LSTM_ACT_GELU_TANH = 3, /* v (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3))) / 2 */
    LSTM_ACT_SILU = 4       /* v / (1 + e^-v) */
};

#define LSTM_DENSE_MAX (1 << 29)

/* y[r][n] = act(sum_k x[r][k] * w[n][k] + bias[n]) + residual[r][n]
 *   x        : device [rows][in]
 *   w        : device [out][in] of x's type, row stride w_stride
 *   bias     : device [out] fp32, or NULL
 *   residual : device [rows][out] of x's type, or NULL; may be y
 *   y        : device [rows][out]
 *   workspace: as lstm_linear_attention's; lstm_dense_workspace(...) bytes
 * rows, in and out are at most LSTM_DENSE_MAX.
 * Sums are the tensor cores', in fp32 and cut off below their last bit (up to
 * three rows: fp32's).  With LSTM_F32 factors go as three parts of bf16: a product
 * loses 2^-24 of itself at most, and what of its factors lies below 2^-133.
 * LSTM_ACT_GELU's factor is good to 2^-20 of itself, however small (16-bit types:
 * 2^-16).
 * 16-bit x and w whose rows all start on 16-byte boundaries are read in place, and
 * so is everything up to three rows; others, and fp32, go through the workspace
 * first.
 * An infinity or a NaN in x or w, and a product beyond fp32, give what fp32 sums
 * give, infinite or NaN.  A wait inside the kernel that does not end within two
 * seconds (and what a sum over K takes) sets the fault word as
 * lstm_linear_attention's.
 * Errors: LSTM_E_INVALID, LSTM_E_LENGTH (workspace), LSTM_E_OVERFLOW,
 * LSTM_E_DEVICE, LSTM_E_CUDA. */
size_t lstm_dense_workspace(const void *x, long long x_stride, const void *w, long long w_stride,
                            int dtype, int rows, int in, int out);
int lstm_dense(const void *x, long long x_stride, const void *w, long long w_stride,
               const float *bias, int activation, const void *residual, long long residual_stride,
               int dtype, int rows, int in, int out, void *y, long long y_stride, void *workspace,
               size_t workspace_bytes, void *stream);

/* Failure-injection hooks, as lstm_test_recurrence_timeout: with withhold != 0
 * lstm_linear_attention and lstm_dense load nothing, so that their waits run out. */
int lstm_test_attention_timeout(int withhold, unsigned int wait_limit_us, int device);
int lstm_test_dense_timeout(int withhold, unsigned int wait_limit_us, int device);

#ifdef __cplusplus
}
#endif

#endif /* LSTM_LAYERS_H */
