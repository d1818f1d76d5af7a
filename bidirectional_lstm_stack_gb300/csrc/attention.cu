// Linear attention with a decay for each head, per sequence and head
//     S_t = e^(g_t) S_(t-1) + k_t v_t^T,   y_t = scale S_t^T q_t:
// the entry points.  attention_prompts.cuh has the prompts' kernels (one file for each
// element type instantiates them), attention_step.cu the single tokens'.
#include "attention.cuh"

namespace lstm {
namespace {

// ---- spans ------------------------------------------------------------------------------
constexpr int kChunk = 64;   // tokens that the prompts' kernel takes at a time
constexpr int kSms = 152;    // one block of it on each
constexpr int kLeastSpan = 4;  // chunks
// In times of a chunk: what a span's chunk costs beside one of a whole sequence, since its
// update is made twice; what starting a block costs, twice too; the two further launches;
// and joining one head's state of one span (128 x 128: written and read twice).
constexpr double kSpanCost = 1.65, kStartCost = 6.0, kLaunchCost = 2.0, kJoinCost = 0.01;

// Chunks of a span, or 0: sequences are whole.  With few sequences and heads most SMs
// would idle, and with sequences of unequal length (the longest taken to be twice the mean)
// the longest would be waited for.
int span_chunks(int tokens, int heads, int values, int sequences, bool equal_lengths)
{
    if (tokens <= 0 || sequences <= 0)
        return 0;
    const double blocks = static_cast<double>(heads) * ((values + 127) / 128);
    const double all = blocks * sequences;
    if (all > 4 * kSms)
        return 0;
    const long long mean = ((tokens - 1LL) / sequences + 1 + kChunk - 1) / kChunk;
    const auto turns = [](double units) {
        return static_cast<double>((static_cast<long long>(units) + kSms - 1) / kSms);
    };
    const double longest = static_cast<double>(equal_lengths ? mean : 2 * mean);
    double best = longest > turns(all) * mean ? longest : turns(all) * mean;
    int chunks = 0;
    for (long long spans = 2; spans <= 64 && mean / spans >= kLeastSpan; ++spans) {
        const long long each = (mean + spans - 1) / spans;
        const double cost = turns(all * spans) * (each * kSpanCost + kStartCost) + kLaunchCost +
                            kJoinCost * all * spans;
        if (cost < best) {
            best = cost;
            chunks = static_cast<int>(each);
        }
    }
    return chunks;
}

// The spans of a call, without their buffers; their bytes.
Spans plan_spans(int tokens, int heads, int keys, int values, int sequences, bool equal_lengths,
                 size_t *bytes)
{
    Spans r;
    r.tokens = span_chunks(tokens, heads, values, sequences, equal_lengths) * kChunk;
    *bytes = 0;
    if (r.tokens) {
        r.units = static_cast<int>(tiles_bound(tokens, sequences, r.tokens));
        *bytes = static_cast<size_t>(r.units) * heads * (static_cast<size_t>(keys) * values + 1) * 4;
    }
    return r;
}

// From what each span adds to a state of zeros to the states that the spans start from: a
// thread takes V numbers of a head's state along a sequence's spans.  All it reads are
// states once, and it writes them once.
constexpr int kJoinThreads = 128;
constexpr int kJoinAhead = 4;  // spans in flight

template <int V>
__global__ void __launch_bounds__(kJoinThreads) attention_join_kernel(const AttentionArgs p,
                                                                      const Spans spans)
{
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int sequence = blockIdx.z, head = blockIdx.y;
    const long long at = (blockIdx.x * static_cast<long long>(kJoinThreads) + threadIdx.x) * V;
    const int begin = sequence_begin(p.seq, sequence);
    const int count = spans.count(sequence_end(p.seq, sequence) - begin);
    if (count == 1 || at >= p.cells())
        return;
    const int unit = begin / spans.tokens + sequence;
    const int slot = sequence_slot(p.slots, sequence);
    Pack<float, V> s = {};
    if (slot >= 0 && sequence_resumes(p.slots, sequence)) {
        const float *from = p.state_of(slot, head) + at;
#pragma unroll
        for (int i = 0; i < V; ++i)
            s.v[i] = from[i];
        *reinterpret_cast<Pack<float, V> *>(spans.state_of(p, unit, head) + at) = s;
    }
    for (int n = 1; n < count; n += kJoinAhead) {
        Pack<float, V> add[kJoinAhead];
        float left[kJoinAhead];
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k)
            if (n + k < count) {
                add[k] = *reinterpret_cast<const Pack<float, V> *>(
                    spans.state_of(p, unit + n + k, head) + at);
                left[k] = *spans.left_of(p, unit + n + k - 1, head);
            }
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k)
            if (n + k < count) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    s.v[i] = fmaf(left[k], s.v[i], add[k].v[i]);
                *reinterpret_cast<Pack<float, V> *>(spans.state_of(p, unit + n + k, head) + at) = s;
            }
    }
}

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
    size_t bytes = 0;
    Spans spans;
    if (!step) {
        spans = plan_spans(rows, p.heads, p.keys, p.values, p.seq.count, !p.seq.offsets, &bytes);
        if (bytes > 0 && !workspace)
            return fail(LSTM_E_INVALID, "%s: workspace is null", what);
        if (workspace_bytes < bytes)
            return fail(LSTM_E_LENGTH, "%s: workspace has %zu bytes, needs %zu", what,
                        workspace_bytes, bytes);
        if ((st = check_aligned(workspace, "workspace")))
            return st;
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
    spans.states = static_cast<float *>(workspace);
    spans.left = spans.states + static_cast<size_t>(spans.units) * p.heads * p.keys * p.values;
    return dtype == LSTM_F32    ? launch_attention_f32(p, spans, on)
           : dtype == LSTM_BF16 ? launch_attention_bf16(p, spans, on)
                                : launch_attention_f16(p, spans, on);
}

}  // namespace

int launch_attention_join(const AttentionArgs &p, const Spans &spans, cudaStream_t stream)
{
    const int st = check_launch_injection("lstm_linear_attention");
    if (st != LSTM_OK)
        return st;
    const long long cells = static_cast<long long>(p.keys) * p.values;
    const int vector = cells % 4 == 0 ? 4 : 1;
    // (sequences that are cut are few)
    const dim3 grid(static_cast<unsigned>((cells + kJoinThreads * vector - 1) / (kJoinThreads * vector)),
                    static_cast<unsigned>(p.heads), static_cast<unsigned>(p.seq.count));
    Dependent launch(grid, kJoinThreads, 0, stream);
    return cuda_status(vector == 4
                           ? cudaLaunchKernelEx(&launch.config, attention_join_kernel<4>, p, spans)
                           : cudaLaunchKernelEx(&launch.config, attention_join_kernel<1>, p, spans),
                       "lstm_linear_attention launch");
}

}  // namespace lstm

using namespace lstm;

extern "C" size_t lstm_linear_attention_workspace(int tokens, int heads, int keys, int values,
                                                  int sequences, int equal_lengths)
{
    if (heads <= 0 || heads > LSTM_ATTENTION_MAX_HEADS || keys <= 0 || keys > LSTM_ATTENTION_MAX_KEYS ||
        values <= 0 || values > LSTM_ATTENTION_MAX_VALUES || tokens > kMostTokens)
        return 0;
    size_t bytes;
    plan_spans(tokens, heads, keys, values, sequences, equal_lengths != 0, &bytes);
    return bytes;
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
