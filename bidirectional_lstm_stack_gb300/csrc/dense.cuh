// What the files of the dense product share.
#pragma once

#include "lstm_layers.h"
#include "ops.cuh"

namespace lstm {

// Up to here rows go without the tensor cores (dense_few.cu).
constexpr int kFewestRows = 3;

struct FewArgs {
    const void *x, *w;
    const float *bias;
    const void *residual;
    void *y;
    long long x_stride, w_stride, residual_stride, y_stride;
    int rows, in, out;
    int activation;
};
int launch_dense_few(const FewArgs &p, int dtype, cudaStream_t stream);

#ifdef __CUDACC__
__device__ __forceinline__ float activate(int kind, float v)
{
    switch (kind) {
    case LSTM_ACT_RELU:
        return v < 0.0f ? 0.0f : v;  // (NaN stays)
    case LSTM_ACT_GELU: {
        // v Phi(v), with erfc(x) = (a1 t + .. + a5 t^5) e^(-x^2), t = 1 / (1 + p x), off by
        // 1.5e-7 at most (Abramowitz and Stegun, 7.1.26): twelve instructions, where both
        // branches of erff take some fifty
        const float x = fabsf(v) * 0.70710678118654752f;
        const float t = reciprocal(fmaf(0.3275911f, x, 1.0f));
        float h = fmaf(t, 1.061405429f, -1.453152027f);
        h = fmaf(t, h, 1.421413741f);
        h = fmaf(t, h, -0.284496736f);
        h = fmaf(t, h, 0.254829592f);
        h = 0.5f * t * h * ex2(-kLog2e * x * x);
        return v * (v < 0.0f ? h : 1.0f - h);
    }
    case LSTM_ACT_GELU_TANH: {
        // (1 + tanh z) / 2 = 1 / (1 + e^-2z): an exponential and a quotient, where tanhf takes
        // some forty instructions; where z is minus infinity the product is -0
        const float z = 0.7978845608028654f * fmaf(0.044715f * v * v, v, v);
        return v * reciprocal(1.0f + ex2(-2.0f * kLog2e * z));
    }
    case LSTM_ACT_SILU:
        return silu(v);
    default:
        return v;
    }
}
#endif

}  // namespace lstm
