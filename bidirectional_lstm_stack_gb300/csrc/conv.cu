// Short causal depthwise convolution over packed prompts, and over the next
// token of each sequence.
//
//   y[t][d] = act(bias[d] + sum_k w[d][k] x[t - (W-1) + k][d]),  W <= 4
//
// Memory-bound: a token's channel costs 2 W + 5 operations and moves two
// elements.  A thread owns four neighbouring channels (or two or one, where
// rows are not aligned) and a run of RUN tokens: it slides the window through
// registers, so each input is loaded once but for the W - 1 rows that a run
// reads from the one before it.  Runs never cross sequences, and a sequence's
// first run is the only reader of its old state and the writer of its new one,
// so a state can be updated in place.
//
// 12288 tokens x 4096 channels of bf16 in 24 prompts: 37 us, 5.4 TB/s of the
// inputs and outputs, 80 % of the card's copy rate; 4096 x 4096, which the L2
// holds, 13.3.  What bounds it now is as much the instructions (without the
// activation 36 and 11.5 us).  With rows loaded four ahead into registers
// instead of a ring in shared memory, and conditions at every token, they
// took 44 and 17.
#include "ops.cuh"

namespace lstm {
namespace {

constexpr int kGroup = 4;  // tokens loaded and worked on together
// Rows of a thread's ring; all but kGroup of them are on their way while it
// works, 57 KB an SM of 16-bit types (12288 x 4096 bf16 37.4 us, 32 x 589 x 256
// fp32 5.4; with 8 rows 38.1 and 5.7).
constexpr int kRing = 12;
// A thread's channels: four (of fp32 16 bytes, of 16-bit types 8).  Eight would
// take 128 registers and leave a quarter of the threads (12288 x 4096 bf16,
// before the ring: 44 us with four, 57 with eight).
constexpr int kVector = 4;
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

// A thread's channels as it works on them: pairs, or the single one.
template <int V>
struct Lane {
    static constexpr int kCount = V / 2;
    typedef Pair Value;
    static __device__ __forceinline__ Pair value(const float *p, int stride)
    {
        return make_pair(p[0], p[stride]);
    }
    static __device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c) { return fma2(a, b, c); }
    static __device__ __forceinline__ void act(Pair (&v)[kCount]) { silu_pairs(v); }
    static __device__ __forceinline__ void split(Pair p, float *f)
    {
        const float2 v = split_pair(p);
        f[0] = v.x;
        f[1] = v.y;
    }
};
template <>
struct Lane<1> {
    static constexpr int kCount = 1;
    typedef float Value;
    static __device__ __forceinline__ float value(const float *p, int) { return p[0]; }
    static __device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
    static __device__ __forceinline__ void act(float (&v)[1]) { v[0] = silu(v[0]); }
    static __device__ __forceinline__ void split(float v, float *f) { f[0] = v; }
};
template <int V>
constexpr int kWide = V > 1 ? 2 : 1;  // channels of a Value

template <typename T, int V>
__device__ __forceinline__ void read(const Pack<T, V> &p,
                                     typename Lane<V>::Value (&v)[Lane<V>::kCount])
{
    float f[V];
    unpack<T, V>(p, f);
#pragma unroll
    for (int i = 0; i < Lane<V>::kCount; ++i)
        v[i] = Lane<V>::value(f + i * kWide<V>, 1);
}

template <int V, int W>
struct Taps {
    typename Lane<V>::Value w[W][Lane<V>::kCount];
    typename Lane<V>::Value bias[Lane<V>::kCount];
};
template <int V, int W>
__device__ __forceinline__ void load_taps(const ConvArgs &a, int d, Taps<V, W> &taps)
{
    float w[V * W], bias[V] = {};
    const float *from = a.w + static_cast<long long>(d) * W;
    if constexpr (V > 1) {
        load_weights<V * W>(from, w);
    } else {
        // taken for weights at any element as well, so no vector of a channel's taps
#pragma unroll
        for (int k = 0; k < W; ++k)
            w[k] = __ldg(from + k);
    }
    if (a.bias)
        load_weights<V>(a.bias + d, bias);
#pragma unroll
    for (int i = 0; i < Lane<V>::kCount; ++i) {
#pragma unroll
        for (int k = 0; k < W; ++k)
            taps.w[k][i] = Lane<V>::value(w + i * kWide<V> * W + k, W);
        taps.bias[i] = Lane<V>::value(bias + i * kWide<V>, 1);
    }
}

// The output of the window x[0..W-1].
template <typename T, int V, int W>
__device__ __forceinline__ Pack<T, V> convolve(
    const typename Lane<V>::Value (&x)[W][Lane<V>::kCount], const Taps<V, W> &taps, bool act)
{
    typename Lane<V>::Value acc[Lane<V>::kCount];
#pragma unroll
    for (int i = 0; i < Lane<V>::kCount; ++i)
        acc[i] = taps.bias[i];
#pragma unroll
    for (int k = 0; k < W; ++k)
#pragma unroll
        for (int i = 0; i < Lane<V>::kCount; ++i)
            acc[i] = Lane<V>::fma(taps.w[k][i], x[k][i], acc[i]);
    if (act)
        Lane<V>::act(acc);
    float f[V];
#pragma unroll
    for (int i = 0; i < Lane<V>::kCount; ++i)
        Lane<V>::split(acc[i], f + i * kWide<V>);
    return pack<T, V>(f);
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

template <typename T, int V>
__device__ __forceinline__ void copy_async(Pack<T, V> *dst, const T *src)
{
    if constexpr (sizeof(Pack<T, V>) == 16)
        ptx::cp_async_16(ptx::smem_u32(dst), src, 16);
    else if constexpr (sizeof(Pack<T, V>) == 8)
        ptx::cp_async_8(ptx::smem_u32(dst), src, 8);
    else
        ptx::cp_async_4(ptx::smem_u32(dst), src, 4);
}

// grid (tiles / blockDim.y, channel vectors / blockDim.x): thread (x, y) of a
// block takes the channel vector x and the run y.
template <typename T, int V, int W, int RUN, bool SILU>
__global__ void __launch_bounds__(kThreads, 7) conv_kernel(ConvArgs a, int tiles)
{
    const int d = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    const int number = blockIdx.x * blockDim.y + threadIdx.y;
    if (d >= a.channels || number >= tiles)
        return;
    Taps<V, W> taps;
    load_taps(a, d, taps);
    int tile;
    const int s = tile_owner(a.seq, number, RUN, &tile);
    const int begin = sequence_begin(a.seq, s), length = sequence_end(a.seq, s) - begin;
    const int t0 = tile * RUN;
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
    typename Lane<V>::Value line[W][Lane<V>::kCount];
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
        read<T, V>(window[k], line[k]);
    const int end = min(t0 + RUN, length);
    x += t0 * a.x_stride;
    y += t0 * a.y_stride;
    // One output, of the row given; the window moves on.
    const auto token = [&](const Pack<T, V> &row) {
        read<T, V>(row, line[W - 1]);
        store_pack<T, V>(y, convolve<T, V, W>(line, taps, SILU));
        y += a.y_stride;
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
#pragma unroll
            for (int i = 0; i < Lane<V>::kCount; ++i)
                line[k][i] = line[k + 1][i];
    };
    if constexpr (sizeof(Pack<T, V>) >= 4) {
        // Rows come through a ring of the thread's own places in shared memory,
        // which holds more of them than registers could: no barriers, and a
        // place is written again only after the row in it has been used.
        constexpr int kRows = RUN < kRing ? RUN : kRing;
        __shared__ Pack<T, V> ring[kRows][kThreads];
        const int me = threadIdx.y * blockDim.x + threadIdx.x;
        int fetched = t0, into = 0, from = 0;
        const auto fetch = [&] {
            const int left = end - fetched;
            if (left >= kGroup) {
#pragma unroll
                for (int j = 0; j < kGroup; ++j) {
                    copy_async(&ring[into + j][me], x);
                    x += a.x_stride;
                }
            } else {
#pragma unroll 1
                for (int j = 0; j < left; ++j) {
                    copy_async(&ring[into + j][me], x);
                    x += a.x_stride;
                }
            }
            ptx::cp_async_commit();
            fetched += kGroup;
            into = into + kGroup < kRows ? into + kGroup : 0;
        };
#pragma unroll
        for (int g = 1; g < kRows / kGroup; ++g)
            fetch();
#pragma unroll 1
        for (int t = t0; t < end; t += kGroup) {
            fetch();
            ptx::cp_async_wait<kRows / kGroup - 1>();
            if (t + kGroup <= end) {
                Pack<T, V> rows[kGroup];
#pragma unroll
                for (int j = 0; j < kGroup; ++j)
                    rows[j] = ring[from + j][me];
#pragma unroll
                for (int j = 0; j < kGroup; ++j)
                    token(rows[j]);
            } else {
#pragma unroll 1
                for (int j = 0; t + j < end; ++j)
                    token(ring[from + j][me]);
            }
            from = from + kGroup < kRows ? from + kGroup : 0;
        }
    } else {
        // (no asynchronous copy is this small) the next rows are loaded before
        // the present ones are worked on
        Pack<T, V> rows[kGroup], next[kGroup];
#pragma unroll
        for (int j = 0; j < kGroup; ++j)
            if (t0 + j < end)
                rows[j] = load_pack<T, V>(x + j * a.x_stride);
#pragma unroll 1
        for (int t = t0; t < end; t += kGroup) {
            x += kGroup * a.x_stride;
#pragma unroll
            for (int j = 0; j < kGroup; ++j)
                if (t + kGroup + j < end)
                    next[j] = load_pack<T, V>(x + j * a.x_stride);
#pragma unroll
            for (int j = 0; j < kGroup; ++j)
                if (t + j < end)
                    token(rows[j]);
#pragma unroll
            for (int j = 0; j < kGroup; ++j)
                rows[j] = next[j];
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
    Taps<V, W> taps;
    load_taps(a, d, taps);
    typename Lane<V>::Value line[W][Lane<V>::kCount];
#pragma unroll
    for (int k = 0; k < W; ++k)
        read<T, V>(window[k], line[k]);
    if (state) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            store_pack<T, V>(state + static_cast<long long>(k) * a.channels, window[k + 1]);
    }
    store_pack<T, V>(static_cast<T *>(a.y) + static_cast<long long>(s) * a.y_stride + d,
                     convolve<T, V, W>(line, taps, a.silu));
}

template <typename T, int V, int W, int RUN>
int launch_run(const ConvArgs &a, cudaStream_t stream)
{
    const int vectors = (a.channels + V - 1) / V;
    const long long tiles = tiles_bound(a.seq.tokens, a.seq.count, RUN);
    // a row's vectors in equal parts of at most kThreads, and of narrow rows
    // several runs to a block, so that its threads have work
    const int columns = (vectors + kThreads - 1) / kThreads;
    const int across = (vectors + columns - 1) / columns;
    const dim3 block(across, kThreads / across);
    const long long grid = (tiles + block.y - 1) / block.y;
    if (tiles > 0x7fffffffll || columns > 65535)
        return fail(LSTM_E_OVERFLOW, "lstm_causal_conv: %d tokens, %d sequences, %d channels",
                    a.seq.tokens, a.seq.count, a.channels);
    const int st = check_launch_injection("lstm_causal_conv");
    if (st != LSTM_OK)
        return st;
    const auto kernel = a.silu ? conv_kernel<T, V, W, RUN, true> : conv_kernel<T, V, W, RUN, false>;
    kernel<<<dim3(static_cast<unsigned>(grid), columns), block, 0, stream>>>(
        a, static_cast<int>(tiles));
    return cuda_status(cudaGetLastError(), "lstm_causal_conv launch");
}

template <typename T, int V, int W>
int launch(const ConvArgs &a, bool step, cudaStream_t stream)
{
    const int vectors = (a.channels + V - 1) / V;
    if (step) {
        const long long blocks =
            (static_cast<long long>(vectors) * a.seq.count + kThreads - 1) / kThreads;
        if (blocks > 0x7fffffffll)
            return fail(LSTM_E_OVERFLOW, "lstm_causal_conv_step: %d sequences of %d channels",
                        a.seq.count, a.channels);
        const int st = check_launch_injection("lstm_causal_conv_step");
        if (st != LSTM_OK)
            return st;
        conv_step_kernel<T, V, W><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a);
        return cuda_status(cudaGetLastError(), "lstm_causal_conv_step launch");
    }
    // Long runs find their sequence and read the rows before them less often;
    // short ones make more threads where there is little to do.  Measured in
    // bf16, runs of 32, 16 and 4 tokens (64): 12288 x 4096 37, 42 and 79 us (38),
    // 4096 x 4096 13.4, 14.6 and 25 us (14.4), 2048 x 2048 5.6, 5.1 and 6.7 us
    // (6.9), 512 x 1024 4.5, 3.5 and 2.9 us (6.6); between 16 and 4 1024 x 2048
    // 4.1 and 4.4 us, 1024 x 1024 3.8 and 3.3 us.
    const long long vector_tokens = static_cast<long long>(vectors) * a.seq.tokens;
    if (vector_tokens >= 1 << 21)
        return launch_run<T, V, W, 32>(a, stream);
    if (vector_tokens >= 1 << 19)
        return launch_run<T, V, W, 16>(a, stream);
    return launch_run<T, V, W, 4>(a, stream);
}

template <typename T, int V>
int launch_width(const ConvArgs &a, int width, bool step, cudaStream_t stream)
{
    switch (width) {
    case 2:
        return launch<T, V, 2>(a, step, stream);
    case 3:
        return launch<T, V, 3>(a, step, stream);
    default:
        return launch<T, V, 4>(a, step, stream);
    }
}

template <typename T>
int launch_typed(const ConvArgs &a, int width, bool step, cudaStream_t stream)
{
    const int size = sizeof(T);
    // whole vectors where every row of x, y and the states, and the weights,
    // start on one; else pairs of 16-bit channels, the least that an asynchronous
    // copy takes; else a channel at a time, with nothing on more than an element's
    // boundary (8192 rows of bf16: 2044 channels 14 us,
    // 2046 15 us in pairs and 24 singly, 2047 24 us)
    const auto fits = [&](int v) {
        return a.channels % v == 0 && (reinterpret_cast<uintptr_t>(a.w) & 15) == 0 &&
               (v < 4 || (reinterpret_cast<uintptr_t>(a.bias) & 15) == 0) &&
               rows_aligned(a.x, a.x_stride, size, v * size) &&
               rows_aligned(a.y, a.y_stride, size, v * size) &&
               (!a.state || rows_aligned(a.state, a.channels, size, v * size));
    };
    if (fits(kVector))
        return launch_width<T, kVector>(a, width, step, stream);
    if constexpr (sizeof(T) == 2)
        if (fits(2))
            return launch_width<T, 2>(a, width, step, stream);
    return launch_width<T, 1>(a, width, step, stream);
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
    const int st = check_sequences("lstm_causal_conv_step", sequences, sequences, nullptr);
    if (st != LSTM_OK)
        return st;
    ConvArgs a = {x, x_stride, w, bias, y, y_stride, state, {nullptr, sequences, 1, sequences},
                  {slots, nullptr, state_slots}, channels, silu != 0};
    return conv("lstm_causal_conv_step", a, dtype, sequences, width, true, stream);
}
