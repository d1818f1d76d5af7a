// Selective state space scan over packed prompts, and over the next token of
// each sequence.
//
//   h[n] = e^(s a[n]) h[n] + s u b[t][n],   v = sum_n h[n] c[t][n] + skip u
//
// per channel, with s the step size of that token and channel and the states
// h in fp32 registers from the first token to the last.
#include "ops.cuh"

namespace lstm {
namespace {

struct ScanArgs {
    const void *u;
    long long u_stride;
    const void *dt;
    long long dt_stride;
    const float *a;
    const void *b;
    long long b_stride;
    const void *c;
    long long c_stride;
    const float *skip;
    const void *z;
    long long z_stride;
    const float *dt_bias;
    int softplus;
    int channels;
    int states;
    int groups;
    float *state;
    Sequences seq;
    Slots slots;
    void *y;
    long long y_stride;
};

// log(1 + e^v) = max(v, 0) + log(1 + e^-|v|); with e = e^-|v| in (0, 1] and
// r = e / (2 + e) <= 1/3, log(1 + e) = 2 atanh(r) = 2 (r + r^3/3 + r^5/5 + ...):
// the series to r^13 leaves less than 2^-26 of the value for every e, where
// log(1 + e) computed as written loses its small values to the sum's rounding.
__device__ __forceinline__ float softplus(float v)
{
    const float e = ex2(-kLog2e * fabsf(v));
    const float r = __fdividef(e, 2.0f + e);
    const float q = r * r;
    float p = fmaf(q, 1.0f / 13.0f, 1.0f / 11.0f);
    p = fmaf(p, q, 1.0f / 9.0f);
    p = fmaf(p, q, 1.0f / 7.0f);
    p = fmaf(p, q, 1.0f / 5.0f);
    p = fmaf(p, q, 1.0f / 3.0f);
    p = fmaf(p, q, 1.0f);
    return fmaf(2.0f * r, p, fmaxf(v, 0.0f));
}

constexpr int kThreads = 128;
constexpr int kStates = 16;  // states a thread holds
constexpr int kTile = 16;    // tokens whose b and c are staged together

// grid (channel blocks of a group * groups, sequences).  G lanes share a
// channel, each with kStates of its states.
template <typename T, int G>
__global__ void __launch_bounds__(kThreads) scan_kernel(ScanArgs p)
{
    constexpr int kPadded = kStates * G;
    __shared__ __align__(16) float sb[kTile][kPadded], sc[kTile][kPadded];
    const int per_group = p.channels / p.groups;
    const int blocks = (per_group + kThreads / G - 1) / (kThreads / G);
    const int group = blockIdx.x / blocks;
    const int local = (blockIdx.x % blocks) * (kThreads / G) + threadIdx.x / G;
    const bool live = local < per_group;
    const int d = group * per_group + (live ? local : 0);
    const int n0 = threadIdx.x % G * kStates;
    const int s = blockIdx.y;
    const int begin = sequence_begin(p.seq, s), end = sequence_end(p.seq, s);
    const int slot = sequence_slot(p.slots, s);
    float *state = slot < 0 ? nullptr
                            : p.state + (static_cast<long long>(slot) * p.channels + d) * p.states;
    const bool resumes = state && sequence_resumes(p.slots, s);
    float h[kStates], a[kStates];
#pragma unroll
    for (int n = 0; n < kStates; ++n) {
        const bool in = n0 + n < p.states;
        h[n] = resumes && in ? state[n0 + n] : 0.0f;
        a[n] = in ? kLog2e * __ldg(p.a + static_cast<long long>(d) * p.states + n0 + n) : 0.0f;
    }
    const float skip = p.skip ? __ldg(p.skip + d) : 0.0f;
    const float dt_bias = p.dt_bias ? __ldg(p.dt_bias + d) : 0.0f;
    const T *u = static_cast<const T *>(p.u) + d;
    const T *dt = static_cast<const T *>(p.dt) + d;
    const T *z = p.z ? static_cast<const T *>(p.z) + d : nullptr;
    const T *b = static_cast<const T *>(p.b) + group * p.states;
    const T *c = static_cast<const T *>(p.c) + group * p.states;
    T *y = static_cast<T *>(p.y) + d;
    for (int t0 = begin; t0 < end; t0 += kTile) {
        const int count = min(kTile, end - t0);
        __syncthreads();
        for (int i = threadIdx.x; i < kTile * kPadded; i += kThreads) {
            const int t = i / kPadded, n = i % kPadded;
            const bool in = t < count && n < p.states;
            sb[t][n] = in ? Elem<T>::get(b[(t0 + t) * p.b_stride + n]) : 0.0f;
            sc[t][n] = in ? Elem<T>::get(c[(t0 + t) * p.c_stride + n]) : 0.0f;
        }
        __syncthreads();
        for (int t = 0; t < count; ++t) {
            const float ut = Elem<T>::get(u[(t0 + t) * p.u_stride]);
            float st = Elem<T>::get(dt[(t0 + t) * p.dt_stride]) + dt_bias;
            if (p.softplus)
                st = softplus(st);
            const float su = st * ut;
            float v = 0.0f;
#pragma unroll
            for (int n = 0; n < kStates; ++n) {
                h[n] = fmaf(ex2(st * a[n]), h[n], su * sb[t][n0 + n]);
                v = fmaf(h[n], sc[t][n0 + n], v);
            }
#pragma unroll
            for (int m = 1; m < G; m <<= 1)
                v += __shfl_xor_sync(0xffffffffu, v, m);
            if (live && n0 == 0) {
                v = fmaf(skip, ut, v);
                if (z)
                    v *= silu(Elem<T>::get(z[(t0 + t) * p.z_stride]));
                y[(t0 + t) * p.y_stride] = Elem<T>::put(v);
            }
        }
    }
    if (state && live) {
#pragma unroll
        for (int n = 0; n < kStates; ++n)
            if (n0 + n < p.states)
                state[n0 + n] = h[n];
    }
}

// ---- single tokens -------------------------------------------------------------
// Memory-bound: the states are read and written once, 8 bytes a state against
// some eight operations.  A thread owns four states of a channel (16 bytes,
// so that a warp's accesses are whole consecutive lines) and L lanes a channel.
template <typename T, int L, bool WIDE>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(ScanArgs p)
{
    const long long at = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) / L;
    const bool live = at < static_cast<long long>(p.seq.count) * p.channels;
    const int s = live ? static_cast<int>(at / p.channels) : 0;
    const int d = live ? static_cast<int>(at % p.channels) : 0;
    const int n0 = threadIdx.x % L * 4;
    const int group = d / (p.channels / p.groups);
    const int slot = sequence_slot(p.slots, s);
    float *state = slot < 0 ? nullptr
                            : p.state + (static_cast<long long>(slot) * p.channels + d) * p.states;
    const float *ap = p.a + static_cast<long long>(d) * p.states;
    const T *b = static_cast<const T *>(p.b) + s * p.b_stride + group * p.states;
    const T *c = static_cast<const T *>(p.c) + s * p.c_stride + group * p.states;
    float h[4] = {}, a[4] = {}, bn[4] = {}, cn[4] = {};
    if (WIDE) {
        if (n0 < p.states) {
            *reinterpret_cast<float4 *>(a) = __ldg(reinterpret_cast<const float4 *>(ap + n0));
            if (state)
                *reinterpret_cast<float4 *>(h) = *reinterpret_cast<const float4 *>(state + n0);
        }
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        if (n0 + n < p.states) {
            if (!WIDE) {
                a[n] = __ldg(ap + n0 + n);
                h[n] = state ? state[n0 + n] : 0.0f;
            }
            bn[n] = Elem<T>::get(b[n0 + n]);
            cn[n] = Elem<T>::get(c[n0 + n]);
        }
    }
    const float ut = Elem<T>::get(static_cast<const T *>(p.u)[s * p.u_stride + d]);
    float st = Elem<T>::get(static_cast<const T *>(p.dt)[s * p.dt_stride + d]);
    if (p.dt_bias)
        st += __ldg(p.dt_bias + d);
    if (p.softplus)
        st = softplus(st);
    const float su = st * ut;
    float v = 0.0f;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        h[n] = fmaf(ex2(st * (kLog2e * a[n])), h[n], su * bn[n]);
        v = fmaf(h[n], cn[n], v);
    }
#pragma unroll
    for (int m = 1; m < L; m <<= 1)
        v += __shfl_xor_sync(0xffffffffu, v, m);
    if (!live)
        return;
    if (state) {
        if (WIDE) {
            if (n0 < p.states)
                *reinterpret_cast<float4 *>(state + n0) = *reinterpret_cast<float4 *>(h);
        } else {
#pragma unroll
            for (int n = 0; n < 4; ++n)
                if (n0 + n < p.states)
                    state[n0 + n] = h[n];
        }
    }
    if (n0 == 0) {
        if (p.skip)
            v = fmaf(__ldg(p.skip + d), ut, v);
        if (p.z)
            v *= silu(Elem<T>::get(static_cast<const T *>(p.z)[s * p.z_stride + d]));
        static_cast<T *>(p.y)[s * p.y_stride + d] = Elem<T>::put(v);
    }
}

template <typename T, int L>
int launch_step(const ScanArgs &p, cudaStream_t stream)
{
    const long long blocks =
        (static_cast<long long>(p.seq.count) * p.channels * L + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffll)
        return fail(LSTM_E_OVERFLOW, "lstm_selective_scan_step: %d sequences, %d channels",
                    p.seq.count, p.channels);
    const int st = check_launch_injection("lstm_selective_scan_step");
    if (st != LSTM_OK)
        return st;
    // whole quads where each channel's states start on a 16-byte boundary
    if (p.states % 4 == 0 && rows_aligned(p.state, p.states, 4) && rows_aligned(p.a, p.states, 4))
        scan_step_kernel<T, L, true><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p);
    else
        scan_step_kernel<T, L, false><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p);
    return cuda_status(cudaGetLastError(), "lstm_selective_scan_step launch");
}

template <typename T, int G>
int launch_prompts(const ScanArgs &p, cudaStream_t stream)
{
    const int per_group = p.channels / p.groups;
    const long long blocks =
        static_cast<long long>((per_group + kThreads / G - 1) / (kThreads / G)) * p.groups;
    if (p.seq.count > 65535 || blocks > 0x7fffffffll)
        return fail(LSTM_E_OVERFLOW, "lstm_selective_scan: %d sequences, %d channels", p.seq.count,
                    p.channels);
    const int st = check_launch_injection("lstm_selective_scan");
    if (st != LSTM_OK)
        return st;
    scan_kernel<T, G><<<dim3(static_cast<unsigned>(blocks), p.seq.count), kThreads, 0, stream>>>(p);
    return cuda_status(cudaGetLastError(), "lstm_selective_scan launch");
}

template <typename T>
int launch_typed(const ScanArgs &p, bool step, cudaStream_t stream)
{
    if (step) {
        if (p.states <= 4)
            return launch_step<T, 1>(p, stream);
        if (p.states <= 8)
            return launch_step<T, 2>(p, stream);
        if (p.states <= 16)
            return launch_step<T, 4>(p, stream);
        if (p.states <= 32)
            return launch_step<T, 8>(p, stream);
        if (p.states <= 64)
            return launch_step<T, 16>(p, stream);
        return launch_step<T, 32>(p, stream);
    }
    if (p.states <= kStates)
        return launch_prompts<T, 1>(p, stream);
    if (p.states <= 2 * kStates)
        return launch_prompts<T, 2>(p, stream);
    if (p.states <= 4 * kStates)
        return launch_prompts<T, 4>(p, stream);
    return launch_prompts<T, 8>(p, stream);
}

int scan(const char *what, ScanArgs &p, int dtype, int rows, bool step, void *stream)
{
    int st;
    if ((st = check_dtype(what, dtype)))
        return st;
    if (rows < 0 || p.channels <= 0 || p.states <= 0 || p.states > LSTM_SCAN_MAX_STATES ||
        p.groups <= 0 || p.channels % p.groups)
        return fail(LSTM_E_INVALID, "%s: %d rows, %d channels, %d states (1 to %d), %d groups", what,
                    rows, p.channels, p.states, LSTM_SCAN_MAX_STATES, p.groups);
    const int size = element_size(dtype);
    const long long wide = static_cast<long long>(p.groups) * p.states;
    if (rows > 0 &&  // without rows there may be no buffers either
        ((st = check_matrix(what, "u", p.u, p.u_stride, rows, p.channels, size)) ||
         (st = check_matrix(what, "dt", p.dt, p.dt_stride, rows, p.channels, size)) ||
         (st = check_matrix(what, "b", p.b, p.b_stride, rows, wide, size)) ||
         (st = check_matrix(what, "c", p.c, p.c_stride, rows, wide, size)) ||
         (p.z && (st = check_matrix(what, "z", p.z, p.z_stride, rows, p.channels, size))) ||
         (st = check_matrix(what, "y", p.y, p.y_stride, rows, p.channels, size))))
        return st;
    if (!p.a)
        return fail(LSTM_E_INVALID, "%s: a is null", what);
    if (p.state) {
        if (p.slots.count < 0)
            return fail(LSTM_E_INVALID, "%s: %d state slots", what, p.slots.count);
        if ((st = check_matrix(what, "state", p.state, p.states, 1, p.states, 4)))
            return st;
    } else {
        p.slots = Slots{nullptr, nullptr, 0};
    }
    int device = 0;
    if ((st = op_device(p.a, &device)))
        return st;
    if (p.seq.count == 0)
        return LSTM_OK;
    DeviceGuard guard(device);
    if (!guard.ok)
        return fail(LSTM_E_CUDA, "cannot make device %d current", device);
    LSTM_WITH_TYPE(dtype, T, return launch_typed<T>(p, step, static_cast<cudaStream_t>(stream)));
}

}  // namespace
}  // namespace lstm

using namespace lstm;

extern "C" int lstm_selective_scan(const void *u, long long u_stride, const void *dt,
                                   long long dt_stride, const float *a, const void *b,
                                   long long b_stride, const void *c, long long c_stride,
                                   const float *skip, const void *z, long long z_stride,
                                   const float *dt_bias, int softplus, int dtype, int tokens,
                                   int channels, int states, int groups, int sequences,
                                   const int *offsets, float *state, int state_slots,
                                   const int *slots, const int *resume, void *y,
                                   long long y_stride, void *stream)
{
    const int st = check_sequences("lstm_selective_scan", tokens, sequences, offsets);
    if (st != LSTM_OK)
        return st;
    ScanArgs p = {u, u_stride, dt, dt_stride, a, b, b_stride, c, c_stride, skip, z, z_stride,
                  dt_bias, softplus != 0, channels, states, groups, state,
                  {offsets, sequences, sequences ? tokens / sequences : 0, tokens},
                  {slots, resume, state_slots}, y, y_stride};
    return scan("lstm_selective_scan", p, dtype, tokens, false, stream);
}

extern "C" int lstm_selective_scan_step(const void *u, long long u_stride, const void *dt,
                                        long long dt_stride, const float *a, const void *b,
                                        long long b_stride, const void *c, long long c_stride,
                                        const float *skip, const void *z, long long z_stride,
                                        const float *dt_bias, int softplus, int dtype,
                                        int sequences, int channels, int states, int groups,
                                        float *state, int state_slots, const int *slots, void *y,
                                        long long y_stride, void *stream)
{
    if (!state)
        return fail(LSTM_E_INVALID, "lstm_selective_scan_step: state is null");
    ScanArgs p = {u, u_stride, dt, dt_stride, a, b, b_stride, c, c_stride, skip, z, z_stride,
                  dt_bias, softplus != 0, channels, states, groups, state,
                  {nullptr, sequences, 1, sequences}, {slots, nullptr, state_slots}, y, y_stride};
    return scan("lstm_selective_scan_step", p, dtype, sequences, true, stream);
}
