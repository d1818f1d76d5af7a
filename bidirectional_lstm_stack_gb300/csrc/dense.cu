// Dense product with bias, activation and residual in its epilogue:
//     y[r][n] = act(sum_k x[r][k] w[n][k] + bias[n]) + residual[r][n].
#include "lstm_layers.h"
#include "ops.cuh"

namespace lstm {
namespace {

struct DenseArgs {
    const void *x, *w;
    long long x_stride, w_stride;
    const float *bias;
    int activation;
    const void *residual;
    long long residual_stride;
    int rows, in, out;
    void *y;
    long long y_stride;
};

__device__ __forceinline__ float activate(int kind, float v)
{
    switch (kind) {
    case LSTM_ACT_RELU:
        return v < 0.0f ? 0.0f : v;  // (NaN stays)
    case LSTM_ACT_GELU:
        return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    case LSTM_ACT_GELU_TANH:
        return 0.5f * v * (1.0f + tanhf(0.7978845608028654f * fmaf(0.044715f * v * v, v, v)));
    case LSTM_ACT_SILU:
        return v / (1.0f + expf(-v));
    default:
        return v;
    }
}

constexpr int kTile = 32;

template <typename T>
__global__ void __launch_bounds__(kTile * 8) dense_kernel(const DenseArgs p)
{
    __shared__ float a[kTile][kTile + 1], b[kTile][kTile + 1];
    const int x = threadIdx.x % kTile, y = threadIdx.x / kTile;
    const long long n0 = static_cast<long long>(blockIdx.x) * kTile;
    for (long long r0 = static_cast<long long>(blockIdx.y) * kTile; r0 < p.rows;
         r0 += static_cast<long long>(gridDim.y) * kTile) {
        float sum[4] = {};
        for (int k0 = 0; k0 < p.in; k0 += kTile) {
            __syncthreads();
            for (int i = y; i < kTile; i += 8) {
                const bool in = x < p.in - k0;
                a[i][x] = in && r0 + i < p.rows
                              ? Elem<T>::get(static_cast<const T *>(p.x)[(r0 + i) * p.x_stride + k0 + x])
                              : 0.0f;
                b[i][x] = in && n0 + i < p.out
                              ? Elem<T>::get(static_cast<const T *>(p.w)[(n0 + i) * p.w_stride + k0 + x])
                              : 0.0f;
            }
            __syncthreads();
            for (int k = 0; k < kTile; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sum[j] = fmaf(a[y + 8 * j][k], b[x][k], sum[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const long long r = r0 + y + 8 * j, n = n0 + x;
            if (r < p.rows && n < p.out) {
                float v = activate(p.activation, sum[j] + (p.bias ? p.bias[n] : 0.0f));
                if (p.residual)
                    v += Elem<T>::get(static_cast<const T *>(p.residual)[r * p.residual_stride + n]);
                static_cast<T *>(p.y)[r * p.y_stride + n] = Elem<T>::put(v);
            }
        }
    }
}

}  // namespace
}  // namespace lstm

using namespace lstm;

extern "C" size_t lstm_dense_workspace(const void *, long long, const void *, long long, int, int,
                                       int, int)
{
    return 0;
}

extern "C" int lstm_dense(const void *x, long long x_stride, const void *w, long long w_stride,
                          const float *bias, int activation, const void *residual,
                          long long residual_stride, int dtype, int rows, int in, int out, void *y,
                          long long y_stride, void *workspace, size_t workspace_bytes, void *stream)
{
    const char *what = "lstm_dense";
    int st;
    if ((st = check_dtype(what, dtype)))
        return st;
    if (rows < 0 || in <= 0 || out <= 0 || activation < LSTM_ACT_NONE || activation > LSTM_ACT_SILU)
        return fail(LSTM_E_INVALID, "%s: %d rows, %d to %d columns, activation %d", what, rows, in,
                    out, activation);
    if (rows > kMostTokens || in > kMostTokens || out > kMostTokens)
        return fail(LSTM_E_OVERFLOW, "%s: %d rows, %d to %d columns (at most %d)", what, rows, in,
                    out, kMostTokens);
    const int size = element_size(dtype);
    if ((st = check_matrix(what, "w", w, w_stride, out, in, size)) ||
        (bias && (st = check_matrix(what, "bias", bias, out, 1, out, 4))))
        return st;
    if (rows > 0 && ((st = check_matrix(what, "x", x, x_stride, rows, in, size)) ||
                     (residual && (st = check_matrix(what, "residual", residual, residual_stride,
                                                     rows, out, size))) ||
                     (st = check_matrix(what, "y", y, y_stride, rows, out, size))))
        return st;
    int device = 0;
    if ((st = op_device(w, &device)))
        return st;
    if (rows == 0)
        return LSTM_OK;
    const size_t needed = lstm_dense_workspace(x, x_stride, w, w_stride, dtype, rows, in, out);
    if (needed > 0 && !workspace)
        return fail(LSTM_E_INVALID, "%s: workspace is null", what);
    if (workspace_bytes < needed)
        return fail(LSTM_E_LENGTH, "%s: workspace has %zu bytes, needs %zu", what, workspace_bytes,
                    needed);
    if ((st = check_aligned(workspace, "workspace")))
        return st;
    DeviceGuard guard(device);
    if (!guard.ok)
        return fail(LSTM_E_CUDA, "cannot make device %d current", device);
    if ((st = check_launch_injection(what)))
        return st;
    const DenseArgs p = {x, w, x_stride, w_stride, bias, activation, residual, residual_stride,
                         rows, in, out, y, y_stride};
    const long long tall = (rows + kTile - 1LL) / kTile;
    const dim3 grid(static_cast<unsigned>((out + kTile - 1LL) / kTile),
                    static_cast<unsigned>(tall < 65535 ? tall : 65535));
    LSTM_WITH_TYPE(dtype, T, (dense_kernel<T><<<grid, kTile * 8, 0,
                                                static_cast<cudaStream_t>(stream)>>>(p)));
    return cuda_status(cudaGetLastError(), "lstm_dense launch");
}
