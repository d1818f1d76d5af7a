// The selective scan's next token of every sequence.
//
// Memory-bound: the states are read and written once, 8 bytes a state against
// some eight operations.  A thread owns four states of a channel (16 bytes,
// so that a warp's accesses are whole consecutive lines) and L lanes a channel.
#include "scan.cuh"

namespace lstm {
namespace {

constexpr int kThreads = 128;

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
    if (p.softplus) {
        Pair v[1] = {make_pair(st, st)};
        softplus_pairs(v);
        st = split_pair(v[0]).x;
    }
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
        if constexpr (WIDE) {
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

template <typename T>
int launch_typed(const ScanArgs &p, cudaStream_t stream)
{
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

}  // namespace

int launch_scan_step(const ScanArgs &p, int dtype, cudaStream_t stream)
{
    LSTM_WITH_TYPE(dtype, T, return launch_typed<T>(p, stream));
}

}  // namespace lstm
