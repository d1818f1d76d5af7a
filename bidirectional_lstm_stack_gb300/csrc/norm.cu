// Residual addition and root-mean-square norm, in the input's type or in 8
// bits (e4m3) with a scale per row or per group of columns.
//
//   v = x + residual,  n = v / sqrt(mean v^2 + eps) * weight
//
// Memory-bound: a handful of operations per element.  One pass: a block holds
// its row in registers between the sum of squares and the outputs, so every
// input is read once and every output written once.  12288 rows of 4096 bf16:
// with a residual to e4m3 and a scale per 128 columns 60 us (5.9 TB/s, 86 % of
// the card's copy rate); 8192 rows to bf16 41 us (6.5 TB/s, 96 %).
#include <cfloat>

#include <cuda_fp8.h>

#include "ops.cuh"

namespace lstm {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr int kMaxCols = 32768;

struct NormArgs {
    const void *x;
    long long x_stride;
    const void *residual;
    long long residual_stride;
    void *residual_out;
    long long residual_out_stride;
    const float *weight;
    float eps;
    void *y;
    long long y_stride;
    float *scales;
    int shift;  // 2^shift columns have a scale; 0: one scale a row
    int groups;
    int cols;
    float mean;  // 1 / cols
};

// The scale of a group whose largest |n| is given: the quotient by 448 as fp32
// rounds it (a product, and one correction by what it leaves; of an infinity
// that is NaN, in whose place fmaxf gives the other number).
__device__ __forceinline__ float e4m3_scale(float most)
{
    constexpr float kInverse = 1.0f / kE4m3Max;
    const float q = most * kInverse, left = fmaxf(fmaf(q, -kE4m3Max, most), -FLT_MAX);
    return most == 0.0f ? 1.0f : fmaxf(fmaf(left, kInverse, q), 0x1p-126f);
}

// What n / scale, as fp32 rounds it, is computed with: the scale's reciprocal in
// two numbers, n / scale = n x + n y.  (By an infinite scale: 0.)
__device__ __forceinline__ float2 e4m3_divisor(float scale)
{
    const float x = reciprocal(scale);
    return make_float2(x, fmaxf(fmaf(-scale, x, 1.0f), -1.0f) * x);
}

// The sum or the largest of a block's values, in every thread.
template <int THREADS, typename F>
__device__ __forceinline__ float block_reduce(float v, float *scratch, F f)
{
    v = warp_reduce(v, f);
    if (threadIdx.x % 32 == 0)
        scratch[threadIdx.x / 32] = v;
    __syncthreads();
    v = scratch[0];
#pragma unroll
    for (int w = 1; w < THREADS / 32; ++w)
        v = f(v, scratch[w]);
    return v;
}

// One row per block; thread t holds the vectors t, t + THREADS, ... (K of
// them).  QUANT: 8-bit output.
template <typename T, int V, int K, int THREADS, bool QUANT>
__global__ void __launch_bounds__(THREADS) norm_kernel(NormArgs p)
{
    __shared__ float scratch[2][THREADS / 32];
    // V == 1: the groups' largest, as float bits in x; then their divisors
    extern __shared__ float2 group_by[];
    const auto sum = [](float a, float b) { return a + b; };
    const auto top = [](float a, float b) { return fmaxf(a, b); };
    const int row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.x_stride;
    const T *res = static_cast<const T *>(p.residual) + row * p.residual_stride;
    T *res_out = static_cast<T *>(p.residual_out) + row * p.residual_out_stride;
    // everything is loaded before anything is stored: residual_out may be
    // residual, so the compiler could not move the loads forward
    Pack<T, V> x_pack[K], res_pack[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * THREADS + threadIdx.x) * V;
        if (c < p.cols) {
            x_pack[k] = load_pack<T, V>(x + c);
            if (p.residual)
                res_pack[k] = *reinterpret_cast<const Pack<T, V> *>(res + c);
        }
    }
    float v[K][V];
    float squares = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * THREADS + threadIdx.x) * V;
        if (c < p.cols) {
            unpack<T, V>(x_pack[k], v[k]);
            if (p.residual) {
                float r[V];
                unpack<T, V>(res_pack[k], r);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    v[k][i] += r[i];
                store_pack<T, V>(res_out + c, pack<T, V>(v[k]));
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[k][i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            squares = fmaf(v[k][i], v[k][i], squares);
    }
    squares = block_reduce<THREADS>(squares, scratch[0], sum);
    const float norm = rsqrtf(fmaf(squares, p.mean, p.eps));
    float most[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * THREADS + threadIdx.x) * V;
        most[k] = 0.0f;
        if (c < p.cols) {
            float w[V];
            load_weights<V>(p.weight + c, w);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[k][i] = v[k][i] * norm * w[i];
                most[k] = fmaxf(most[k], fabsf(v[k][i]));
            }
        }
    }
    if constexpr (!QUANT) {
        T *y = static_cast<T *>(p.y) + row * p.y_stride;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * THREADS + threadIdx.x) * V;
            if (c < p.cols)
                store_pack<T, V>(y + c, pack<T, V>(v[k]));
        }
        return;
    }
    __nv_fp8_storage_t *y = static_cast<__nv_fp8_storage_t *>(p.y) + row * p.y_stride;
    float *scales = p.scales + static_cast<long long>(row) * p.groups;
    if (p.shift == 0) {
#pragma unroll
        for (int k = 1; k < K; ++k)
            most[0] = fmaxf(most[0], most[k]);
        most[0] = block_reduce<THREADS>(most[0], scratch[1], top);
#pragma unroll
        for (int k = 1; k < K; ++k)
            most[k] = most[0];
    } else if (V > 1) {
        // group / V consecutive lanes hold a group
#pragma unroll
        for (int k = 0; k < K; ++k)
            for (int m = (1 << p.shift) / V / 2; m; m >>= 1)
                most[k] = fmaxf(most[k], __shfl_xor_sync(0xffffffffu, most[k], m));
    } else {
        // a warp's 32 columns lie in one group; the order of the maxima does
        // not change the result
        for (int g = threadIdx.x; g < p.groups; g += THREADS)
            group_by[g].x = 0.0f;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float m = warp_reduce(most[k], top);
            const int c = k * THREADS + threadIdx.x;
            if (threadIdx.x % 32 == 0 && c < p.cols)
                atomicMax(reinterpret_cast<unsigned *>(&group_by[c >> p.shift].x), __float_as_uint(m));
        }
        __syncthreads();
        for (int g = threadIdx.x; g < p.groups; g += THREADS) {
            const float scale = e4m3_scale(group_by[g].x);
            scales[g] = scale;
            group_by[g] = e4m3_divisor(scale);
        }
        __syncthreads();
    }
    if constexpr (V == 1) {
        float2 by = {};
        if (p.shift == 0) {
            const float scale = e4m3_scale(most[0]);
            by = e4m3_divisor(scale);
            if (threadIdx.x == 0)
                scales[0] = scale;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = k * THREADS + threadIdx.x;
            if (c >= p.cols)
                continue;
            if (p.shift)
                by = group_by[c >> p.shift];
            y[c] = __nv_cvt_float_to_fp8(fmaf(v[k][0], by.x, v[k][0] * by.y), __NV_SATFINITE,
                                         __NV_E4M3);
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * THREADS + threadIdx.x) * V;
            if (c >= p.cols)
                continue;
            const float scale = e4m3_scale(most[k]);
            const float2 by = e4m3_divisor(scale);
            Pack<__nv_fp8_storage_t, V> q;
            // (paired, so that the second product costs no more issue slots: 12288 x
            // 4096 by groups of 128 60.2 us with the first product alone, 61.6 with
            // both singly, 60.4 in pairs)
            const Pair x = make_pair(by.x, by.x), rest = make_pair(by.y, by.y);
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                const Pair n = make_pair(v[k][i], v[k][i + 1]);
                *reinterpret_cast<__nv_fp8x2_storage_t *>(q.v + i) = __nv_cvt_float2_to_fp8x2(
                    split_pair(fma2(n, x, mul2(n, rest))), __NV_SATFINITE, __NV_E4M3);
            }
            store_pack(y + c, q);
            if (p.shift ? (c & ((1 << p.shift) - 1)) == 0 : c == 0)
                scales[p.shift ? c >> p.shift : 0] = scale;
        }
    }
}

template <typename T, int V, int K, int THREADS>
int launch(const NormArgs &p, int rows, bool quant, cudaStream_t stream)
{
    const int st = check_launch_injection("lstm_residual_rms_norm");
    if (st != LSTM_OK)
        return st;
    const size_t shared = V == 1 && quant && p.shift ? p.groups * sizeof(float2) : 0;
    if (quant)
        norm_kernel<T, V, K, THREADS, true><<<rows, THREADS, shared, stream>>>(p);
    else
        norm_kernel<T, V, K, THREADS, false><<<rows, THREADS, shared, stream>>>(p);
    return cuda_status(cudaGetLastError(), "lstm_residual_rms_norm launch");
}

template <typename T, int V>
int launch_sized(const NormArgs &p, int rows, bool quant, cudaStream_t stream)
{
    const int vectors = (p.cols + V - 1) / V;
    if constexpr (V == 1) {
        // single elements: several a thread (2047 columns of bf16, 8192 rows, to
        // e4m3 by groups: 256 threads of eight 40 us; with the groups' divisors
        // computed for every element 42, 512 of four 50, 1024 of two 80)
        if (vectors <= 512)
            return launch<T, 1, 2, 256>(p, rows, quant, stream);
        if (vectors <= 2048)
            return launch<T, 1, 8, 256>(p, rows, quant, stream);
        if (vectors <= 8192)
            return launch<T, 1, 8, 1024>(p, rows, quant, stream);
        return launch<T, 1, 32, 1024>(p, rows, quant, stream);
    } else {
        // One vector a thread while a block has threads for it: with more,
        // fewer loads are on their way at a time (4096 columns of bf16, 12288
        // rows to e4m3: 512 threads 60 us, 256 of two vectors 68, 128 of four
        // 86).
        if (vectors <= 64)
            return launch<T, V, 1, 64>(p, rows, quant, stream);
        if (vectors <= 128)
            return launch<T, V, 1, 128>(p, rows, quant, stream);
        if (vectors <= 256)
            return launch<T, V, 1, 256>(p, rows, quant, stream);
        if (vectors <= 512)
            return launch<T, V, 1, 512>(p, rows, quant, stream);
        if (vectors <= 1024)
            return launch<T, V, 1, 1024>(p, rows, quant, stream);
        if (vectors <= 2048)
            return launch<T, V, 2, 1024>(p, rows, quant, stream);
        return launch<T, V, kMaxCols / V / 1024, 1024>(p, rows, quant, stream);
    }
}

template <typename T>
int launch_typed(const NormArgs &p, int rows, bool quant, cudaStream_t stream)
{
    constexpr int V = Elem<T>::kVector;
    const int size = sizeof(T);
    // whole vectors where every row of every matrix starts on one; otherwise
    // an element at a time
    const bool wide =
        p.cols % V == 0 && (reinterpret_cast<uintptr_t>(p.weight) & 15) == 0 &&
        rows_aligned(p.x, p.x_stride, size) &&
        (!p.residual || (rows_aligned(p.residual, p.residual_stride, size) &&
                         rows_aligned(p.residual_out, p.residual_out_stride, size))) &&
        (quant ? reinterpret_cast<uintptr_t>(p.y) % V == 0 && p.y_stride % V == 0
               : rows_aligned(p.y, p.y_stride, size));
    return wide ? launch_sized<T, V>(p, rows, quant, stream) : launch_sized<T, 1>(p, rows, quant, stream);
}

}  // namespace
}  // namespace lstm

using namespace lstm;

extern "C" int lstm_residual_rms_norm(const void *x, long long x_stride, const void *residual,
                                      long long residual_stride, int dtype, const float *weight,
                                      float eps, int rows, int cols, void *residual_out,
                                      long long residual_out_stride, void *y, long long y_stride,
                                      int y_dtype, float *scales, int group, void *stream)
{
    const char *what = "lstm_residual_rms_norm";
    int st;
    if ((st = check_dtype(what, dtype)))
        return st;
    const bool quant = y_dtype == LSTM_E4M3;
    if (!quant && y_dtype != dtype)
        return fail(LSTM_E_INVALID, "%s: output type %d (%d, the input's, or %d)", what, y_dtype,
                    dtype, LSTM_E4M3);
    if (rows < 0 || cols <= 0 || cols > kMaxCols)
        return fail(LSTM_E_INVALID, "%s: %d rows, %d columns (1 to %d)", what, rows, cols, kMaxCols);
    if (quant && group != 0 && group != 32 && group != 64 && group != 128)
        return fail(LSTM_E_INVALID, "%s: group %d (0, 32, 64 or 128)", what, group);
    if (!(eps >= 0.0f))
        return fail(LSTM_E_INVALID, "%s: eps %g", what, eps);
    if (!residual != !residual_out)
        return fail(LSTM_E_INVALID, "%s: residual and residual_out go together", what);
    if (!weight)
        return fail(LSTM_E_INVALID, "%s: weight is null", what);
    if (rows == 0)
        return LSTM_OK;
    const int size = element_size(dtype);
    if ((st = check_matrix(what, "x", x, x_stride, rows, cols, size)) ||
        (st = check_matrix(what, "y", y, y_stride, rows, cols, quant ? 1 : size)) ||
        (residual &&
         ((st = check_matrix(what, "residual", residual, residual_stride, rows, cols, size)) ||
          (st = check_matrix(what, "residual_out", residual_out, residual_out_stride, rows, cols,
                             size)))) ||
        (quant && (st = check_matrix(what, "scales", scales, 1, 1, 1, 4))))
        return st;
    int device = 0;
    if ((st = op_device(x, &device)))
        return st;
    DeviceGuard guard(device);
    if (!guard.ok)
        return fail(LSTM_E_CUDA, "cannot make device %d current", device);
    const int shift = !quant ? 0 : group == 32 ? 5 : group == 64 ? 6 : group == 128 ? 7 : 0;
    NormArgs p = {x, x_stride, residual, residual_stride, residual_out, residual_out_stride, weight,
                  eps, y, y_stride, scales, shift, shift ? ((cols - 1) >> shift) + 1 : 1, cols,
                  1.0f / cols};
    LSTM_WITH_TYPE(dtype, T,
                   return launch_typed<T>(p, rows, quant, static_cast<cudaStream_t>(stream)));
}
