// Linear attention with a decay for each head, per sequence and head
//     S_t = e^(g_t) S_(t-1) + k_t v_t^T,   y_t = scale S_t^T q_t:
// the entry points.  attention_prompts.cuh has the prompts' kernels (one file for each
// element type instantiates them), attention_step.cu the single tokens'.
#include "attention.cuh"

namespace lstm {
namespace {

int check_heads(const char *what, const char *name, HeadRows &m, int own, int heads, int width,
                int rows, int size)
{
    if (own <= 0 || heads % own)
        return fail(LSTM_E_INVALID, "%s: %s has %d heads, which do not divide %d", what, name, own,
                    heads);
    m.share = heads / own;
    if (own == 1)
        m.head_stride = 0;
    else if (m.head_stride < width)
        return fail(LSTM_E_INVALID, "%s: %s has heads %lld apart, heads of %d", what, name,
                    m.head_stride, width);
    if (rows == 0)  // without rows there may be no buffers either
        return LSTM_OK;
    return check_matrix(what, name, m.at, m.stride, rows, width, size);
}

int attention(const char *what, AttentionArgs &p, int q_heads, int k_heads, int v_heads, int dtype,
              int rows, bool step, void *workspace, size_t workspace_bytes, void *stream)
{
    int st;
    if ((st = check_dtype(what, dtype)))
        return st;
    if (rows < 0 || p.heads <= 0 || p.heads > LSTM_ATTENTION_MAX_HEADS || p.keys <= 0 ||
        p.keys > LSTM_ATTENTION_MAX_KEYS || p.values <= 0 || p.values > LSTM_ATTENTION_MAX_VALUES)
        return fail(LSTM_E_INVALID,
                    "%s: %d rows, %d heads (1 to %d) of %d keys (1 to %d) and %d values (1 to %d)",
                    what, rows, p.heads, LSTM_ATTENTION_MAX_HEADS, p.keys, LSTM_ATTENTION_MAX_KEYS,
                    p.values, LSTM_ATTENTION_MAX_VALUES);
    const int size = element_size(dtype);
    if ((st = check_heads(what, "q", p.q, q_heads, p.heads, p.keys, rows, size)) ||
        (st = check_heads(what, "k", p.k, k_heads, p.heads, p.keys, rows, size)) ||
        (st = check_heads(what, "v", p.v, v_heads, p.heads, p.values, rows, size)))
        return st;
    if (rows > 0 &&
        (st = check_matrix(what, "y", p.y, p.y_stride, rows,
                           static_cast<long long>(p.heads) * p.values, size)))
        return st;
    if (p.decay_stride != 0 && rows > 1 && p.decay_stride < p.heads)
        return fail(LSTM_E_INVALID, "%s: log_decay has row stride %lld, rows of %d (or 0: one row)",
                    what, p.decay_stride, p.heads);
    const bool no_decay = rows == 0 && p.decay_stride != 0 && !p.decay;
    if (!no_decay && (st = check_matrix(what, "log_decay", p.decay, p.heads, 1, p.heads, 4)))
        return st;
    if (p.state) {
        if (p.slots.count < 0)
            return fail(LSTM_E_INVALID, "%s: %d state slots", what, p.slots.count);
        if ((st = check_matrix(what, "state", p.state, p.values, 1, p.values, 4)))
            return st;
    } else {
        p.slots = Slots{nullptr, nullptr, 0};
    }
    int device = 0;
    if (p.seq.count == 0 || (no_decay && !p.state))
        return LSTM_OK;
    if ((st = op_device(no_decay ? p.state : p.decay, &device)))
        return st;
    DeviceGuard guard(device);
    if (!guard.ok)
        return fail(LSTM_E_CUDA, "cannot make device %d current", device);
    cudaStream_t on = static_cast<cudaStream_t>(stream);
    if (step)
        return launch_attention_step(p, dtype, on);
    return dtype == LSTM_F32    ? launch_attention_f32(p, on)
           : dtype == LSTM_BF16 ? launch_attention_bf16(p, on)
                                : launch_attention_f16(p, on);
}

}  // namespace
}  // namespace lstm

using namespace lstm;

extern "C" size_t lstm_linear_attention_workspace(int, int, int, int, int, int)
{
    return 0;
}

extern "C" int lstm_linear_attention(const void *q, long long q_stride, long long q_head_stride,
                                     int q_heads, const void *k, long long k_stride,
                                     long long k_head_stride, int k_heads, const void *v,
                                     long long v_stride, long long v_head_stride, int v_heads,
                                     const float *log_decay, long long decay_stride, float scale,
                                     int dtype, int tokens, int heads, int keys, int values,
                                     int sequences, const int *offsets, float *state,
                                     int state_slots, const int *slots, const int *resume, void *y,
                                     long long y_stride, void *workspace, size_t workspace_bytes,
                                     void *stream)
{
    const int st = check_sequences("lstm_linear_attention", tokens, sequences, offsets);
    if (st != LSTM_OK)
        return st;
    AttentionArgs p = {{q, q_stride, q_head_stride, 1}, {k, k_stride, k_head_stride, 1},
                       {v, v_stride, v_head_stride, 1}, log_decay, decay_stride, scale, heads, keys,
                       values, state,
                       {offsets, sequences, sequences ? tokens / sequences : 0, tokens},
                       {slots, resume, state_slots}, y, y_stride};
    return attention("lstm_linear_attention", p, q_heads, k_heads, v_heads, dtype, tokens, false,
                     workspace, workspace_bytes, stream);
}

extern "C" int lstm_linear_attention_step(const void *q, long long q_stride,
                                          long long q_head_stride, int q_heads, const void *k,
                                          long long k_stride, long long k_head_stride, int k_heads,
                                          const void *v, long long v_stride,
                                          long long v_head_stride, int v_heads,
                                          const float *log_decay, long long decay_stride,
                                          float scale, int dtype, int sequences, int heads,
                                          int keys, int values, float *state, int state_slots,
                                          const int *slots, void *y, long long y_stride,
                                          void *stream)
{
    if (!state)
        return fail(LSTM_E_INVALID, "lstm_linear_attention_step: state is null");
    const int st = check_sequences("lstm_linear_attention_step", sequences, sequences, nullptr);
    if (st != LSTM_OK)
        return st;
    AttentionArgs p = {{q, q_stride, q_head_stride, 1}, {k, k_stride, k_head_stride, 1},
                       {v, v_stride, v_head_stride, 1}, log_decay, decay_stride, scale, heads, keys,
                       values, state, {nullptr, sequences, 1, sequences},
                       {slots, nullptr, state_slots}, y, y_stride};
    return attention("lstm_linear_attention_step", p, q_heads, k_heads, v_heads, dtype, sequences,
                     true, nullptr, 0, stream);
}
