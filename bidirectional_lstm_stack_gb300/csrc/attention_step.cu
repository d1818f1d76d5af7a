// Linear attention's next token: per sequence and head
//     S = e^g S + k v^T,   y = scale S^T q
// with S, keys x values fp32 numbers, read and written once: 8 bytes for 5
// operations, so the states' traffic is all there is (a sequence of 16 heads of
// 128 x 128 moves 2 MiB; 256 of them 541 MB in 85 us, 94 % of the measured
// 6.8 TB/s).  A block takes a head's S or a tile of its columns.
// A thread keeps one vector of columns and goes down every R-th row, its loads
// issued before their first use; the R partial sums of each column are joined
// through shared memory in a fixed order.
#include "attention.cuh"

namespace lstm {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 8;  // rows of a thread in flight

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) attention_step_kernel(const AttentionArgs p, int tile)
{
    __shared__ float q[LSTM_ATTENTION_MAX_KEYS], k[LSTM_ATTENTION_MAX_KEYS];
    __shared__ float part[kThreads * V];
    const int s = blockIdx.x, head = blockIdx.y;
    // threads: `across` vectors of columns times `groups` groups of rows
    const int across = tile / V, groups = blockDim.x / across;
    const int x = threadIdx.x % across, group = threadIdx.x / across;
    const int col = blockIdx.z * tile + x * V;
    const bool inside = col < p.values;
    const int slot = sequence_slot(p.slots, s);
    const float left = expf(__ldg(p.decay + s * p.decay_stride + head));

    float *state = slot >= 0 ? p.state_of(slot, head) + col : nullptr;
    Pack<float, V> h[kAhead];
    const auto fetch = [&](int n) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int row = n + j * groups;
#pragma unroll
            for (int i = 0; i < V; ++i)
                h[j].v[i] = 0.0f;
            if (state && inside && row < p.keys)
                h[j] = *reinterpret_cast<const Pack<float, V> *>(
                    state + static_cast<long long>(row) * p.values);
        }
    };
    fetch(group);
    for (int n = threadIdx.x; n < p.keys; n += blockDim.x) {
        q[n] = Elem<T>::get(p.q.row<T>(s, head)[n]);
        k[n] = Elem<T>::get(p.k.row<T>(s, head)[n]);
    }
    float v[V], sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        v[i] = inside ? Elem<T>::get(p.v.row<T>(s, head)[col + i]) : 0.0f;
        sum[i] = 0.0f;
    }
    __syncthreads();
    for (int n = group; n < p.keys; n += kAhead * groups) {
        if (n != group)
            fetch(n);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int row = n + j * groups;
            if (row < p.keys) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    h[j].v[i] = fmaf(k[row], v[i], left * h[j].v[i]);
                    sum[i] = fmaf(q[row], h[j].v[i], sum[i]);
                }
                if (state && inside)
                    *reinterpret_cast<Pack<float, V> *>(
                        state + static_cast<long long>(row) * p.values) = h[j];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        part[group * tile + x * V + i] = sum[i];
    __syncthreads();
    for (int c = threadIdx.x; c < tile && blockIdx.z * tile + c < p.values; c += blockDim.x) {
        float y = 0.0f;
        for (int g = 0; g < groups; ++g)
            y += part[g * tile + c];
        p.out<T>(s, head)[blockIdx.z * tile + c] = Elem<T>::put(p.scale * y);
    }
}

template <typename T, int V>
int launch(const AttentionArgs &p, cudaStream_t stream)
{
    // as wide a tile as leaves two blocks an SM, at least 32 columns (128 bytes of a row)
    int tile = V;
    while (tile < p.values)
        tile *= 2;
    const long long blocks = static_cast<long long>(p.seq.count) * p.heads;
    while (tile > 32 && blocks * ((p.values + tile - 1) / tile) < 152 * 2)
        tile /= 2;
    const int across = tile / V;
    int groups = kThreads / across;
    while (groups > 1 && groups >= 2 * p.keys)
        groups /= 2;
    const int st = check_launch_injection("lstm_linear_attention_step");
    if (st != LSTM_OK)
        return st;
    const dim3 grid(static_cast<unsigned>(p.seq.count), static_cast<unsigned>(p.heads),
                    static_cast<unsigned>((p.values + tile - 1) / tile));
    attention_step_kernel<T, V><<<grid, across * groups, 0, stream>>>(p, tile);
    return cuda_status(cudaGetLastError(), "lstm_linear_attention_step launch");
}

}  // namespace

int launch_attention_step(const AttentionArgs &p, int dtype, cudaStream_t stream)
{
    const bool vectors = rows_aligned(p.state, p.values, 4);
    LSTM_WITH_TYPE(dtype, T,
                   return vectors ? launch<T, 4>(p, stream) : launch<T, 1>(p, stream));
}

}  // namespace lstm
