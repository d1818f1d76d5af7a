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

// Two fp32 numbers in one 64-bit register: the paired operations do two
// roundings each in one issue slot.
typedef unsigned long long Pair;
__device__ __forceinline__ Pair make_pair(float x, float y)
{
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 split_pair(Pair p)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b)
{
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c)
{
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ Pair ex2_pair(Pair p)
{
    const float2 v = split_pair(p);
    return make_pair(ex2(v.x), ex2(v.y));
}

// ---- prompts --------------------------------------------------------------------
constexpr int kTile = 16;  // tokens staged together
constexpr int kStep = 4;   // of them computed together

// Spans of `chunk` tokens (chunk tiles, in tile_owner's numbering), and what
// the first pass leaves for the second: per span, channel and state, the
// state after the span when it starts from zeros (the sequence's first span:
// from its own start), and the sum of the span's step sizes.  A sequence's
// last span has nothing to leave; its place holds the state that the sequence
// starts from, which the second pass may not read where it is kept, because
// the last span replaces it.
struct Spans {
    int chunk;
    float *states;  // [numbers][channels][padded]
    float *sums;    // [numbers][channels]
};

template <typename T, int CH, int PADDED, bool GATE>
struct alignas(16) Stage {
    T u[kTile][CH];
    T dt[kTile][CH];
    T z[GATE ? kTile : 1][CH];
    float b[kTile][PADDED];
    float c[GATE ? kTile : 1][PADDED];
};

// grid (span numbers, channel blocks of a group * groups).  G lanes share a
// channel, each with NS of its states.  FINAL false: the first pass, over the
// spans that others follow.
template <typename T, int NS, int G, bool WIDE, bool FINAL>
__global__ void __launch_bounds__(kThreads) scan_kernel(ScanArgs p, Spans w)
{
    constexpr int kChannels = kThreads / G;
    constexpr int kPadded = NS * G;
    constexpr int kFetch = kTile * kPadded / kThreads;  // of b, and of c, a thread's share
    constexpr int V = Elem<T>::kVector;
    extern __shared__ __align__(16) unsigned char shared[];
    typedef Stage<T, kChannels, kPadded, FINAL> StageT;
    StageT *stages = reinterpret_cast<StageT *>(shared);

    if (!FINAL)
        ptx::griddep_launch_dependents();
    const int number = blockIdx.x;
    int span;
    const int s = tile_owner(p.seq, number, w.chunk, &span);
    const int seq_begin = sequence_begin(p.seq, s), seq_end = sequence_end(p.seq, s);
    const int length = seq_end - seq_begin;
    const int spans = length > 0 ? (length - 1) / w.chunk + 1 : 1;  // (one to keep the state)
    if (span < 0 || span >= spans || (!FINAL && spans == 1)) {
        if (FINAL)  // what follows this kernel must not overtake the first pass
            ptx::griddep_wait();
        return;
    }
    const bool last = span == spans - 1;
    const int begin = seq_begin + span * w.chunk;
    const int end = last ? seq_end : begin + w.chunk;

    const int per_group = p.channels / p.groups;
    const int blocks = (per_group + kChannels - 1) / kChannels;
    const int group = blockIdx.y / blocks;
    const int local0 = (blockIdx.y % blocks) * kChannels;
    const int here = min(kChannels, per_group - local0);  // channels of this block
    const int c0 = group * per_group + local0;
    const int ch = threadIdx.x / G;
    const bool live = ch < here;
    const int d = c0 + (live ? ch : 0);
    const int n0 = threadIdx.x % G * NS;
    const int slot = sequence_slot(p.slots, s);
    float *state = slot < 0 ? nullptr
                            : p.state + (static_cast<long long>(slot) * p.channels + d) * p.states;
    const bool resumes = state && sequence_resumes(p.slots, s);
    const long long first = number - span;  // the sequence's first span number
    float *kept = w.states + (static_cast<long long>(number) * p.channels + d) * kPadded + n0;

    Pair h[NS / 2], a[NS / 2];
    const float *from = p.a + static_cast<long long>(d) * p.states;
#pragma unroll
    for (int n = 0; n < NS; n += 2) {
        const int k = n0 + n;
        a[n / 2] = make_pair(k < p.states ? kLog2e * __ldg(from + k) : 0.0f,
                             k + 1 < p.states ? kLog2e * __ldg(from + k + 1) : 0.0f);
        h[n / 2] = 0;
    }
    const auto start_from_state = [&]() {
#pragma unroll
        for (int n = 0; n < NS; n += 2) {
            const int k = n0 + n;
            h[n / 2] = make_pair(k < p.states ? state[k] : 0.0f,
                                 k + 1 < p.states ? state[k + 1] : 0.0f);
        }
    };
    if (!FINAL && last) {  // nothing follows: keep the sequence's start
        if (resumes && live) {
            start_from_state();
#pragma unroll
            for (int n = 0; n < NS / 2; n += 2)
                *reinterpret_cast<ulonglong2 *>(kept + 2 * n) = make_ulonglong2(h[n], h[n + 1]);
        }
        return;
    }

    // staging: u, dt and z as they are, asynchronously; b and c as fp32
    const T *u = static_cast<const T *>(p.u) + c0;
    const T *dt = static_cast<const T *>(p.dt) + c0;
    const T *z = FINAL && p.z ? static_cast<const T *>(p.z) + c0 : nullptr;
    const T *b = static_cast<const T *>(p.b) + group * p.states;
    const T *c = static_cast<const T *>(p.c) + group * p.states;
    T fetch_b[kFetch], fetch_c[kFetch];
    const auto fetch = [&](int t0, StageT &st) {
        const int count = min(kTile, end - t0);
        if (WIDE) {
            constexpr int kRow = kChannels / V > 0 ? kChannels / V : 1;
            for (int i = threadIdx.x; i < count * kRow; i += kThreads) {
                const int t = i / kRow, at = i % kRow * V;
                if (at < here) {
                    ptx::cp_async_16(ptx::smem_u32(&st.u[t][at]), u + (t0 + t) * p.u_stride + at, 16);
                    ptx::cp_async_16(ptx::smem_u32(&st.dt[t][at]), dt + (t0 + t) * p.dt_stride + at,
                                     16);
                    if (z)
                        ptx::cp_async_16(ptx::smem_u32(&st.z[t][at]), z + (t0 + t) * p.z_stride + at,
                                         16);
                }
            }
            ptx::cp_async_commit();
        } else {
            for (int i = threadIdx.x; i < count * kChannels; i += kThreads) {
                const int t = i / kChannels, at = i % kChannels;
                if (at < here) {
                    st.u[t][at] = u[(t0 + t) * p.u_stride + at];
                    st.dt[t][at] = dt[(t0 + t) * p.dt_stride + at];
                    if (z)
                        st.z[t][at] = z[(t0 + t) * p.z_stride + at];
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kFetch; ++k) {
            const int i = k * kThreads + threadIdx.x, t = i / kPadded, n = i % kPadded;
            const bool in = t < count && n < p.states;
            fetch_b[k] = in ? b[(t0 + t) * p.b_stride + n] : Elem<T>::put(0.0f);
            if (FINAL)
                fetch_c[k] = in ? c[(t0 + t) * p.c_stride + n] : Elem<T>::put(0.0f);
        }
    };
    const auto settle = [&](StageT &st) {
#pragma unroll
        for (int k = 0; k < kFetch; ++k) {
            const int i = k * kThreads + threadIdx.x, t = i / kPadded, n = i % kPadded;
            st.b[t][n] = Elem<T>::get(fetch_b[k]);
            if (FINAL)
                st.c[t][n] = Elem<T>::get(fetch_c[k]);
        }
        if (WIDE)
            ptx::cp_async_wait_all();
        __syncthreads();
    };

    int stage = 0;
    if (begin < end)
        fetch(begin, stages[0]);
    const float skip = p.skip ? __ldg(p.skip + d) : 0.0f;
    const float dt_bias = p.dt_bias ? __ldg(p.dt_bias + d) : 0.0f;
    T *y = FINAL ? static_cast<T *>(p.y) + d : nullptr;
    if (FINAL)
        ptx::griddep_wait();
    if (FINAL && spans > 1) {
        // the state that this span starts from: every earlier span carries
        // the state before it on by e^(a * its step sizes' sum)
        if (span == 0) {
            if (resumes) {
                const float *start =
                    w.states + ((first + spans - 1) * p.channels + d) * kPadded + n0;
#pragma unroll
                for (int n = 0; n < NS; n += 2)
                    h[n / 2] = *reinterpret_cast<const Pair *>(start + n);
            }
        } else {
            const float *sum = w.sums + first * p.channels + d;
            const float *left = w.states + (first * p.channels + d) * kPadded + n0;
            for (int k = 0; k < span; ++k) {
                const float total = *sum;
                const Pair by = make_pair(total, total);
#pragma unroll
                for (int n = 0; n < NS; n += 2)
                    h[n / 2] = fma2(ex2_pair(mul2(by, a[n / 2])), h[n / 2],
                                    *reinterpret_cast<const Pair *>(left + n));
                sum += p.channels;
                left += static_cast<long long>(p.channels) * kPadded;
            }
        }
    } else if (resumes && span == 0) {
        start_from_state();
    }

    float sum = 0.0f;
    for (int t0 = begin; t0 < end; t0 += kTile) {
        StageT &st = stages[stage];
        settle(st);
        if (t0 + kTile < end)
            fetch(t0 + kTile, stages[stage ^ 1]);
        stage ^= 1;
        const int count = min(kTile, end - t0);
#pragma unroll 1
        for (int t = 0; t < count; t += kStep) {
            float step[kStep], add[kStep], in[kStep];
#pragma unroll
            for (int j = 0; j < kStep; ++j) {
                const bool real = t + j < count;  // (others change nothing)
                in[j] = Elem<T>::get(st.u[t + j][ch]);
                float v = Elem<T>::get(st.dt[t + j][ch]) + dt_bias;
                if (p.softplus)
                    v = softplus(v);
                step[j] = real ? v : 0.0f;
                add[j] = real ? v * in[j] : 0.0f;
                sum += step[j];
            }
#pragma unroll
            for (int j = 0; j < kStep; ++j) {
                const Pair by = make_pair(step[j], step[j]), plus = make_pair(add[j], add[j]);
                Pair out = 0;
#pragma unroll
                for (int n = 0; n < NS / 2; n += 2) {
                    const ulonglong2 bn = *reinterpret_cast<const ulonglong2 *>(&st.b[t + j][n0 + 2 * n]);
                    h[n] = fma2(ex2_pair(mul2(by, a[n])), h[n], mul2(plus, bn.x));
                    h[n + 1] = fma2(ex2_pair(mul2(by, a[n + 1])), h[n + 1], mul2(plus, bn.y));
                    if (FINAL) {
                        const ulonglong2 cn =
                            *reinterpret_cast<const ulonglong2 *>(&st.c[t + j][n0 + 2 * n]);
                        out = fma2(h[n], cn.x, out);
                        out = fma2(h[n + 1], cn.y, out);
                    }
                }
                if (FINAL) {
                    const float2 halves = split_pair(out);
                    float v = halves.x + halves.y;
#pragma unroll
                    for (int m = 1; m < G; m <<= 1)
                        v += __shfl_xor_sync(0xffffffffu, v, m);
                    v = fmaf(skip, in[j], v);
                    if (z)
                        v *= silu(Elem<T>::get(st.z[t + j][ch]));
                    if (t + j < count && live && n0 == 0)
                        y[(t0 + t + j) * p.y_stride] = Elem<T>::put(v);
                }
            }
        }
    }
    if (!live)
        return;
    if (!FINAL) {
#pragma unroll
        for (int n = 0; n < NS / 2; n += 2)
            *reinterpret_cast<ulonglong2 *>(kept + 2 * n) = make_ulonglong2(h[n], h[n + 1]);
        if (n0 == 0)
            w.sums[static_cast<long long>(number) * p.channels + d] = sum;
    } else if (last && state) {
#pragma unroll
        for (int n = 0; n < NS; n += 2) {
            const float2 v = split_pair(h[n / 2]);
            if (n0 + n < p.states)
                state[n0 + n] = v.x;
            if (n0 + n + 1 < p.states)
                state[n0 + n + 1] = v.y;
        }
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

// How a call's prompts are worked on: the same for its workspace's size and
// for its launches.
struct Plan {
    int states;       // a thread's
    int lanes;        // a channel's
    int chunk;        // tokens of a span
    long long spans;  // span numbers
    bool split;       // whether a sequence may have several spans
    size_t bytes;     // of workspace
};

Plan make_plan(int tokens, int channels, int states, int sequences, bool equal)
{
    Plan r;
    r.states = states <= 8 ? 8 : 16;
    r.lanes = 1;
    while (r.states * r.lanes < states)
        r.lanes *= 2;
    // Splitting sequences into spans reads them twice and takes their
    // exponentials twice, so it pays where the sequences alone leave the
    // machine empty.
    const long long threads = static_cast<long long>(channels) * r.lanes;
    const long long wanted = 152 * 256;
    long long chunk = tokens;
    if (sequences * threads < wanted) {
        chunk = tokens * threads / wanted;
        chunk = (chunk + kTile - 1) / kTile * kTile;
        if (chunk < 2 * kTile)
            chunk = 2 * kTile;
    }
    const long long longest = equal ? tokens / (sequences > 0 ? sequences : 1) : tokens;
    r.split = chunk < longest;
    // whole sequences: spans longer than all tokens together number just them
    r.chunk = r.split ? static_cast<int>(chunk) : tokens + 1;
    r.spans = r.split ? tiles_bound(tokens, sequences, r.chunk) : sequences;
    r.bytes = r.split ? static_cast<size_t>(r.spans) * channels * (r.states * r.lanes + 1) * 4 : 0;
    return r;
}

template <typename T, int NS, int G, bool WIDE>
int launch_prompts(const ScanArgs &p, const Plan &plan, void *workspace, cudaStream_t stream)
{
    constexpr int kChannels = kThreads / G;
    const int per_group = p.channels / p.groups;
    const long long blocks =
        static_cast<long long>((per_group + kChannels - 1) / kChannels) * p.groups;
    if (plan.spans > 0x7fffffffll || blocks > 65535)
        return fail(LSTM_E_OVERFLOW, "lstm_selective_scan: %d sequences, %d tokens, %d channels",
                    p.seq.count, p.seq.tokens, p.channels);
    Spans w = {plan.chunk, static_cast<float *>(workspace), nullptr};
    w.sums = w.states + plan.spans * p.channels * NS * G;
    const dim3 grid(static_cast<unsigned>(plan.spans), static_cast<unsigned>(blocks));
    constexpr size_t kShared = 2 * sizeof(Stage<T, kChannels, NS * G, true>);
    constexpr size_t kSharedFirst = 2 * sizeof(Stage<T, kChannels, NS * G, false>);
    static SharedMemory allowed, allowed_first;
    int st;
    if ((st = allowed.allow(scan_kernel<T, NS, G, WIDE, true>, kShared)) ||
        (st = allowed_first.allow(scan_kernel<T, NS, G, WIDE, false>, kSharedFirst)))
        return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    if (plan.split) {
        if ((st = check_launch_injection("lstm_selective_scan")))
            return st;
        cfg.dynamicSmemBytes = kSharedFirst;
        if ((st = cuda_status(cudaLaunchKernelEx(&cfg, scan_kernel<T, NS, G, WIDE, false>, p, w),
                              "lstm_selective_scan launch")))
            return st;
    }
    if ((st = check_launch_injection("lstm_selective_scan")))
        return st;
    cfg.dynamicSmemBytes = kShared;
    // the second pass may start while the first one ends; it waits for it
    // before it reads what that left
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = plan.split ? 1 : 0;
    return cuda_status(cudaLaunchKernelEx(&cfg, scan_kernel<T, NS, G, WIDE, true>, p, w),
                       "lstm_selective_scan launch");
}

template <typename T, int NS, int G>
int launch_aligned(const ScanArgs &p, const Plan &plan, void *workspace, cudaStream_t stream)
{
    constexpr int V = Elem<T>::kVector;
    const int size = sizeof(T);
    // 16-byte copies where every row of u, dt and z, and every group of
    // channels, starts on a 16-byte boundary
    const bool wide = p.channels / p.groups % V == 0 && rows_aligned(p.u, p.u_stride, size) &&
                      rows_aligned(p.dt, p.dt_stride, size) &&
                      (!p.z || rows_aligned(p.z, p.z_stride, size));
    return wide ? launch_prompts<T, NS, G, true>(p, plan, workspace, stream)
                : launch_prompts<T, NS, G, false>(p, plan, workspace, stream);
}

template <typename T>
int launch_typed(const ScanArgs &p, bool step, const Plan &plan, void *workspace,
                 cudaStream_t stream)
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
    if (plan.states == 8)
        return launch_aligned<T, 8, 1>(p, plan, workspace, stream);
    switch (plan.lanes) {
    case 1:
        return launch_aligned<T, 16, 1>(p, plan, workspace, stream);
    case 2:
        return launch_aligned<T, 16, 2>(p, plan, workspace, stream);
    case 4:
        return launch_aligned<T, 16, 4>(p, plan, workspace, stream);
    default:
        return launch_aligned<T, 16, 8>(p, plan, workspace, stream);
    }
}

int scan(const char *what, ScanArgs &p, int dtype, int rows, bool step, void *workspace,
         size_t workspace_bytes, void *stream)
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
    Plan plan = {};
    if (!step) {
        plan = make_plan(rows, p.channels, p.states, p.seq.count, !p.seq.offsets);
        if (plan.bytes > 0 && !workspace)
            return fail(LSTM_E_INVALID, "%s: workspace is null", what);
        if (workspace_bytes < plan.bytes)
            return fail(LSTM_E_LENGTH, "%s: workspace has %zu bytes, needs %zu", what,
                        workspace_bytes, plan.bytes);
        if ((st = check_aligned(workspace, "workspace")))
            return st;
    }
    DeviceGuard guard(device);
    if (!guard.ok)
        return fail(LSTM_E_CUDA, "cannot make device %d current", device);
    LSTM_WITH_TYPE(dtype, T, return launch_typed<T>(p, step, plan, workspace,
                                                    static_cast<cudaStream_t>(stream)));
}

}  // namespace
}  // namespace lstm

using namespace lstm;

extern "C" size_t lstm_selective_scan_workspace(int tokens, int channels, int states, int sequences,
                                                int equal_lengths)
{
    if (tokens <= 0 || channels <= 0 || states <= 0 || states > LSTM_SCAN_MAX_STATES ||
        sequences <= 0)
        return 0;
    return make_plan(tokens, channels, states, sequences, equal_lengths != 0).bytes;
}

extern "C" int lstm_selective_scan(const void *u, long long u_stride, const void *dt,
                                   long long dt_stride, const float *a, const void *b,
                                   long long b_stride, const void *c, long long c_stride,
                                   const float *skip, const void *z, long long z_stride,
                                   const float *dt_bias, int softplus, int dtype, int tokens,
                                   int channels, int states, int groups, int sequences,
                                   const int *offsets, float *state, int state_slots,
                                   const int *slots, const int *resume, void *y,
                                   long long y_stride, void *workspace, size_t workspace_bytes,
                                   void *stream)
{
    const int st = check_sequences("lstm_selective_scan", tokens, sequences, offsets);
    if (st != LSTM_OK)
        return st;
    ScanArgs p = {u, u_stride, dt, dt_stride, a, b, b_stride, c, c_stride, skip, z, z_stride,
                  dt_bias, softplus != 0, channels, states, groups, state,
                  {offsets, sequences, sequences ? tokens / sequences : 0, tokens},
                  {slots, resume, state_slots}, y, y_stride};
    return scan("lstm_selective_scan", p, dtype, tokens, false, workspace, workspace_bytes,
                stream);
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
    return scan("lstm_selective_scan_step", p, dtype, sequences, true, nullptr, 0, stream);
}
