// Short causal depthwise convolution over packed prompts, and over the next
// token of each sequence.
//
//   y[t][d] = act(bias[d] + sum_k w[d][k] x[t - (W-1) + k][d]),  W <= 4
//
// Memory-bound: a token's channel costs 2 W + 5 operations and moves two
// elements.  A thread owns the channels of one 16-byte vector (or one
// channel, where rows are not 16-byte aligned) and a run of kRun tokens: it
// slides the window through registers, so each input is loaded once but for
// the W - 1 rows that a run reads from the one before it.  Runs never cross
// sequences, and a sequence's first run is the only reader of its old state
// and the writer of its new one, so a state can be updated in place.
#include "ops.cuh"

namespace lstm {
namespace {

constexpr int kRun = 16;    // tokens a thread convolves
constexpr int kAhead = 8;   // of them loaded together
constexpr int kThreads = 128;

struct ConvArgs {
    const void *x;
    long long x_stride;
    const float *w;
    const float *bias;
    void *y;
    long long y_stride;
    void *state;
    Sequences seq;
    Slots slots;
    int channels;
    int silu;
};

template <int V, int W>
__device__ __forceinline__ void load_weights(const ConvArgs &a, int d, float (&w)[W][V],
                                             float (&bias)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int k = 0; k < W; ++k)
            w[k][i] = __ldg(a.w + static_cast<long long>(d + i) * W + k);
        bias[i] = a.bias ? __ldg(a.bias + d + i) : 0.0f;
    }
}

// The output of the window x[0..W-1].
template <typename T, int V, int W>
__device__ __forceinline__ Pack<T, V> convolve(const Pack<T, V> (&x)[W], const float (&w)[W][V],
                                               const float (&bias)[V], bool act)
{
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        acc[i] = bias[i];
#pragma unroll
    for (int k = 0; k < W; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i)
            acc[i] = fmaf(w[k][i], Elem<T>::get(x[k].v[i]), acc[i]);
    if (act) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            acc[i] = silu(acc[i]);
    }
    return pack<T, V>(acc);
}

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> zeros()
{
    Pack<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i)
        r.v[i] = Elem<T>::put(0.0f);
    return r;
}

// grid (tiles / blockDim.y, channel vectors / blockDim.x): thread (x, y) of a
// block takes the channel vector x and the run y.
template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads) conv_kernel(ConvArgs a, int tiles)
{
    const int d = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    const int number = blockIdx.x * blockDim.y + threadIdx.y;
    if (d >= a.channels || number >= tiles)
        return;
    int tile;
    const int s = tile_owner(a.seq, number, kRun, &tile);
    const int begin = sequence_begin(a.seq, s), length = sequence_end(a.seq, s) - begin;
    const int t0 = tile * kRun;
    if (tile < 0 || (t0 >= length && tile > 0))
        return;
    const T *x = static_cast<const T *>(a.x) + static_cast<long long>(begin) * a.x_stride + d;
    T *y = static_cast<T *>(a.y) + static_cast<long long>(begin) * a.y_stride + d;
    Pack<T, V> window[W];  // window[0..W-2]: the rows before the next one
    if (tile == 0) {
        const int slot = sequence_slot(a.slots, s);
        T *state = slot < 0 ? nullptr
                            : static_cast<T *>(a.state) +
                                  static_cast<long long>(slot) * (W - 1) * a.channels + d;
        const bool resumes = state && sequence_resumes(a.slots, s);
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            window[k] = resumes ? *reinterpret_cast<const Pack<T, V> *>(state + static_cast<long long>(k) * a.channels)
                                : zeros<T, V>();
        if (state) {
            // the last W - 1 of the old state's rows followed by the sequence's
#pragma unroll
            for (int k = 0; k < W - 1; ++k) {
                const int row = length - (W - 1) + k;
                Pack<T, V> v = zeros<T, V>();
                if (row >= 0) {
                    v = load_pack<T, V>(x + row * a.x_stride);
                } else {
#pragma unroll
                    for (int j = 0; j < W - 1; ++j)
                        if (j == row + W - 1)
                            v = window[j];
                }
                store_pack<T, V>(state + static_cast<long long>(k) * a.channels, v);
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            window[k] = load_pack<T, V>(x + (t0 - (W - 1) + k) * a.x_stride);
    }
    float w[W][V], bias[V];
    load_weights<V, W>(a, d, w, bias);
    const int end = min(t0 + kRun, length);
    for (int t = t0; t < end; t += kAhead) {
        Pack<T, V> next[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (t + j < end)
                next[j] = load_pack<T, V>(x + (t + j) * a.x_stride);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (t + j >= end)
                break;
            window[W - 1] = next[j];
            store_pack<T, V>(y + (t + j) * a.y_stride, convolve<T, V, W>(window, w, bias, a.silu));
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
                window[k] = window[k + 1];
        }
    }
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(ConvArgs a)
{
    const int vectors = (a.channels + V - 1) / V;
    const long long at = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
    const int s = static_cast<int>(at / vectors);
    if (s >= a.seq.count)
        return;
    const int d = static_cast<int>(at % vectors) * V;
    const int slot = sequence_slot(a.slots, s);
    T *state = slot < 0 ? nullptr
                        : static_cast<T *>(a.state) +
                              static_cast<long long>(slot) * (W - 1) * a.channels + d;
    Pack<T, V> window[W];
    window[W - 1] =
        load_pack<T, V>(static_cast<const T *>(a.x) + static_cast<long long>(s) * a.x_stride + d);
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
        window[k] = state ? *reinterpret_cast<const Pack<T, V> *>(state + static_cast<long long>(k) * a.channels)
                          : zeros<T, V>();
    float w[W][V], bias[V];
    load_weights<V, W>(a, d, w, bias);
    if (state) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            store_pack<T, V>(state + static_cast<long long>(k) * a.channels, window[k + 1]);
    }
    store_pack<T, V>(static_cast<T *>(a.y) + static_cast<long long>(s) * a.y_stride + d,
                     convolve<T, V, W>(window, w, bias, a.silu));
}

template <typename T, int V, int W>
int launch(const ConvArgs &a, bool step, cudaStream_t stream)
{
    const int vectors = (a.channels + V - 1) / V;
    int st;
    if (step) {
        const long long blocks =
            (static_cast<long long>(vectors) * a.seq.count + kThreads - 1) / kThreads;
        if (blocks > 0x7fffffffll)
            return fail(LSTM_E_OVERFLOW, "lstm_causal_conv_step: %d sequences of %d channels",
                        a.seq.count, a.channels);
        if ((st = check_launch_injection("lstm_causal_conv_step")))
            return st;
        conv_step_kernel<T, V, W><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a);
        return cuda_status(cudaGetLastError(), "lstm_causal_conv_step launch");
    }
    const long long tiles = tiles_bound(a.seq.tokens, a.seq.count, kRun);
    // narrow rows: several runs to a block, so that its threads have work
    const int across = vectors >= kThreads ? kThreads : (vectors + 31) / 32 * 32;
    const dim3 block(across, kThreads / across);
    const long long grid = (tiles + block.y - 1) / block.y;
    const int columns = (vectors + across - 1) / across;
    if (tiles > 0x7fffffffll || columns > 65535)
        return fail(LSTM_E_OVERFLOW, "lstm_causal_conv: %d tokens, %d sequences, %d channels",
                    a.seq.tokens, a.seq.count, a.channels);
    if ((st = check_launch_injection("lstm_causal_conv")))
        return st;
    conv_kernel<T, V, W><<<dim3(static_cast<unsigned>(grid), columns), block, 0, stream>>>(
        a, static_cast<int>(tiles));
    return cuda_status(cudaGetLastError(), "lstm_causal_conv launch");
}

template <typename T>
int launch_typed(const ConvArgs &a, int width, bool step, cudaStream_t stream)
{
    constexpr int V = Elem<T>::kVector;
    const int size = sizeof(T);
    // whole vectors where every row of x, y and the states starts on one;
    // otherwise a channel at a time
    const bool wide = a.channels % V == 0 && rows_aligned(a.x, a.x_stride, size) &&
                      rows_aligned(a.y, a.y_stride, size) &&
                      (!a.state || rows_aligned(a.state, a.channels, size));
    switch (width) {
    case 2:
        return wide ? launch<T, V, 2>(a, step, stream) : launch<T, 1, 2>(a, step, stream);
    case 3:
        return wide ? launch<T, V, 3>(a, step, stream) : launch<T, 1, 3>(a, step, stream);
    default:
        return wide ? launch<T, V, 4>(a, step, stream) : launch<T, 1, 4>(a, step, stream);
    }
}

int check_conv(const char *what, ConvArgs &a, int dtype, int rows, int width, int *device)
{
    int st;
    if ((st = check_dtype(what, dtype)))
        return st;
    if (rows < 0 || a.channels <= 0 || width < 2 || width > LSTM_CONV_MAX_WIDTH)
        return fail(LSTM_E_INVALID, "%s: %d rows, %d channels, width %d (2 to %d)", what, rows,
                    a.channels, width, LSTM_CONV_MAX_WIDTH);
    const int size = element_size(dtype);
    if (rows > 0 &&  // without rows there may be no buffers either
        ((st = check_matrix(what, "x", a.x, a.x_stride, rows, a.channels, size)) ||
         (st = check_matrix(what, "y", a.y, a.y_stride, rows, a.channels, size))))
        return st;
    if (!a.w)
        return fail(LSTM_E_INVALID, "%s: w is null", what);
    if (a.state) {
        if (a.slots.count < 0)
            return fail(LSTM_E_INVALID, "%s: %d state slots", what, a.slots.count);
        if ((st = check_matrix(what, "state", a.state, a.channels, a.slots.count, a.channels, size)))
            return st;
    } else {
        a.slots = Slots{nullptr, nullptr, 0};
    }
    return op_device(a.w, device);
}

int conv(const char *what, ConvArgs &a, int dtype, int rows, int width, bool step, void *stream)
{
    int device = 0;
    int st = check_conv(what, a, dtype, rows, width, &device);
    if (st != LSTM_OK)
        return st;
    if (a.seq.count == 0)
        return LSTM_OK;
    DeviceGuard guard(device);
    if (!guard.ok)
        return fail(LSTM_E_CUDA, "cannot make device %d current", device);
    LSTM_WITH_TYPE(dtype, T,
                   return launch_typed<T>(a, width, step, static_cast<cudaStream_t>(stream)));
}

}  // namespace
}  // namespace lstm

using namespace lstm;

extern "C" int lstm_causal_conv(const void *x, long long x_stride, int dtype, int tokens,
                                int channels, int width, const float *w, const float *bias,
                                int silu, int sequences, const int *offsets, void *state,
                                int state_slots, const int *slots, const int *resume, void *y,
                                long long y_stride, void *stream)
{
    const int st = check_sequences("lstm_causal_conv", tokens, sequences, offsets);
    if (st != LSTM_OK)
        return st;
    ConvArgs a = {x, x_stride, w, bias, y, y_stride, state,
                  {offsets, sequences, sequences ? tokens / sequences : 0, tokens},
                  {slots, resume, state_slots}, channels, silu != 0};
    return conv("lstm_causal_conv", a, dtype, tokens, width, false, stream);
}

extern "C" int lstm_causal_conv_step(const void *x, long long x_stride, int dtype, int sequences,
                                     int channels, int width, const float *w, const float *bias,
                                     int silu, void *state, int state_slots, const int *slots,
                                     void *y, long long y_stride, void *stream)
{
    if (!state)
        return fail(LSTM_E_INVALID, "lstm_causal_conv_step: state is null");
    ConvArgs a = {x, x_stride, w, bias, y, y_stride, state, {nullptr, sequences, 1, sequences},
                  {slots, nullptr, state_slots}, channels, silu != 0};
    return conv("lstm_causal_conv_step", a, dtype, sequences, width, true, stream);
}
