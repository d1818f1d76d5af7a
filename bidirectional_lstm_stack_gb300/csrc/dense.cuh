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
// FINE: for results of fp32, else of 16 bits.
template <bool FINE>
__device__ __forceinline__ float activate(int kind, float v)
{
    switch (kind) {
    case LSTM_ACT_RELU:
        return v < 0.0f ? 0.0f : v;  // (NaN stays)
    case LSTM_ACT_GELU: {
        // v Phi(v).  With a = |v|, Phi(-a) = e^(-a^2 / 2) t P(t), t = 1 / (1 + q a): P is a
        // least-maximum fit of the relative error up to a = 13.5, beyond which the result leaves
        // fp32's normal range, made for this file from erfc in 64 bits.  (A difference 1 - |erf|
        // would have no digits left below -5.)  FINE: of degree 8, 3e-8 off, and a^2 / 2 keeps
        // its rounding's rest, which is up to 7e-6 of the exponential; the factor is off by less
        // than 2^-20 of itself.  Else of degree 5, 5e-6 off, which leaves 2^-16: sixteen times
        // finer than fp16's rounding, and 2048 x 2048 x 8192 in bf16 takes 54 us, 58 with the
        // fine one.
        const float a = fminf(fabsf(v), 16.0f);
        const float s = a * a, power = -0.72134752f * s;  // -log2(e) / 2 = -0.7213475 - 9.63e-9
        float h, e = ex2(power);
        if constexpr (FINE) {
            const float t = reciprocal(fmaf(0.34f, a, 1.0f));
            h = fmaf(t, -0.026370253f, 0.14067209f);
            h = fmaf(t, h, -0.27546227f);
            h = fmaf(t, h, 0.20473261f);
            h = fmaf(t, h, -0.046395034f);
            h = fmaf(t, h, 0.11603495f);
            h = fmaf(t, h, 0.115035094f);
            h = fmaf(t, h, 0.13613348f);
            h = fmaf(t, h, 0.13561934f) * t;
            const float rest = fmaf(-0.72134752f, fmaf(a, a, -s),
                                    fmaf(-9.629815e-9f, s, fmaf(-0.72134752f, s, -power)));
            e = fmaf(e, 0.6931472f * rest, e);
        } else {
            const float t = reciprocal(fmaf(0.31f, a, 1.0f));
            h = fmaf(t, -0.07392915f, 0.18045036f);
            h = fmaf(t, h, 0.015744697f);
            h = fmaf(t, h, 0.1334298f);
            h = fmaf(t, h, 0.12044128f);
            h = fmaf(t, h, 0.1238607f) * t;
        }
        h *= e;
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
