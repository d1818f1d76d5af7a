// The dense product for a row or a few:  y[r][n] = act(sum_k x[r][k] w[n][k] + bias[n]) +
// residual[r][n].  w is read once for two operations a number and row, so its traffic is all
// there is (4096 x 4096 of 16 bits: 33.6 MB, 4.9 us at the measured 6.8 TB/s; 8.2 us), and tensor cores
// would only add their set-up: a tile's pipeline has to be filled, its accumulator allocated,
// read and joined.  A warp takes four rows of w over a part of K, all lanes side by side along
// a row, and keeps several vectors a lane in flight; the sums of a row's parts are joined in
// shared memory, in the order of the parts.  x comes from the L1 cache.
#include "dense.cuh"

namespace lstm {
namespace {

// (blocks of 256 threads fill the SMs less evenly: 11 us; two columns a warp: 10 us)
constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kColumns = 4;   // of y, rows of w, a warp takes
constexpr int kEnough = 152 * 16;  // warps; with fewer, rows are shared out among more

template <typename T, int R, int V>
__global__ void __launch_bounds__(kThreads) dense_few_kernel(const FewArgs p, int split)
{
    __shared__ float sums[kWarps][kColumns * R];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = warp % split, own = warp / split, groups = kWarps / split;
    const long long n0 = (blockIdx.x * static_cast<long long>(groups) + own) * kColumns;
    float acc[kColumns][R];
#pragma unroll
    for (int c = 0; c < kColumns; ++c)
#pragma unroll
        for (int r = 0; r < R; ++r)
            acc[c][r] = 0.0f;
    // (columns and rows beyond the last are the last's, and not stored)
    const T *w[kColumns], *x[R];
#pragma unroll
    for (int c = 0; c < kColumns; ++c)
        w[c] = static_cast<const T *>(p.w) +
               (n0 + c < p.out ? n0 + c : p.out - 1) * p.w_stride + lane * V;
#pragma unroll
    for (int r = 0; r < R; ++r)
        x[r] = static_cast<const T *>(p.x) + min(r, p.rows - 1) * p.x_stride + lane * V;
    const auto add = [&](const Pack<T, V> (&wv)[kColumns], const Pack<T, V> (&xv)[R]) {
#pragma unroll
        for (int e = 0; e < V; ++e)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float f = Elem<T>::get(xv[r].v[e]);
#pragma unroll
                for (int c = 0; c < kColumns; ++c)
                    acc[c][r] = fmaf(Elem<T>::get(wv[c].v[e]), f, acc[c][r]);
            }
    };
    constexpr int kStep = 32 * V;
    int k = part * kStep;
#pragma unroll (V * sizeof(T) == 16 ? 2 : 4)
    for (; k + kStep <= p.in; k += split * kStep) {
        Pack<T, V> wv[kColumns], xv[R];
#pragma unroll
        for (int c = 0; c < kColumns; ++c)
            wv[c] = load_pack<T, V>(w[c] + k);
#pragma unroll
        for (int r = 0; r < R; ++r)
            xv[r] = load_pack<T, V>(x[r] + k);
        add(wv, xv);
    }
    if (k < p.in) {  // the last numbers, which are one part's
        Pack<T, V> wv[kColumns], xv[R];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const bool in = k + lane * V + e < p.in;
#pragma unroll
            for (int c = 0; c < kColumns; ++c)
                wv[c].v[e] = in ? w[c][k + e] : Elem<T>::put(0.0f);
#pragma unroll
            for (int r = 0; r < R; ++r)
                xv[r].v[e] = in ? x[r][k + e] : Elem<T>::put(0.0f);
        }
        add(wv, xv);
    }
#pragma unroll
    for (int c = 0; c < kColumns; ++c)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float sum = warp_reduce(acc[c][r], [](float a, float b) { return a + b; });
            if (lane == 0)
                sums[warp][r * kColumns + c] = sum;
        }
    __syncthreads();
    const int i = threadIdx.x;
    if (i >= groups * kColumns * R)
        return;
    const int g = i / (kColumns * R), at = i % (kColumns * R), r = at / kColumns;
    const long long n = (blockIdx.x * static_cast<long long>(groups) + g) * kColumns + at % kColumns;
    if (r >= p.rows || n >= p.out)
        return;
    float v = 0.0f;
    for (int s = 0; s < split; ++s)
        v += sums[g * split + s][at];
    if (p.bias)
        v += __ldg(p.bias + n);
    v = activate<sizeof(T) == 4>(p.activation, v);
    if (p.residual)
        v += Elem<T>::get(static_cast<const T *>(p.residual)[r * p.residual_stride + n]);
    static_cast<T *>(p.y)[r * p.y_stride + n] = Elem<T>::put(v);
}

template <typename T, int R, int V>
int launch(const FewArgs &p, cudaStream_t stream)
{
    const long long groups = (p.out + kColumns - 1LL) / kColumns;
    int split = 1;
    while (split < kWarps && groups * split < kEnough && p.in >= 2LL * split * 32 * V)
        split *= 2;
    const int st = check_launch_injection("lstm_dense");
    if (st != LSTM_OK)
        return st;
    const long long each = kWarps / split;
    dense_few_kernel<T, R, V><<<static_cast<unsigned>((groups + each - 1) / each), kThreads, 0, stream>>>(
        p, split);
    return cuda_status(cudaGetLastError(), "lstm_dense launch");
}

template <typename T, int V>
int launch_rows(const FewArgs &p, cudaStream_t stream)
{
    return p.rows == 1   ? launch<T, 1, V>(p, stream)
           : p.rows == 2 ? launch<T, 2, V>(p, stream)
                         : launch<T, kFewestRows, V>(p, stream);
}

}  // namespace

int launch_dense_few(const FewArgs &p, int dtype, cudaStream_t stream)
{
    const int size = element_size(dtype);
    const bool vectors = rows_aligned(p.x, p.rows > 1 ? p.x_stride : 0, size) &&
                         rows_aligned(p.w, p.out > 1 ? p.w_stride : 0, size);
    LSTM_WITH_TYPE(dtype, T,
                   return vectors ? launch_rows<T, Elem<T>::kVector>(p, stream)
                                  : launch_rows<T, 1>(p, stream));
}

}  // namespace lstm
