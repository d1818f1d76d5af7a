// The selective scan over packed prompts: kernels and launches, instantiated
// by scan_f32.cu, scan_bf16.cu and scan_f16.cu.
#pragma once

#include <type_traits>

#include "scan.cuh"

namespace lstm {
namespace {

constexpr int kStep = 8;  // tokens computed together
// tokens staged together: 16, or 8 in fp32, so that two stages of a block take
// about 32 KB of shared memory
template <typename T>
constexpr int kTile = sizeof(T) == 4 ? 8 : 16;

template <typename T, int CH, int PADDED, bool FINAL>
struct alignas(16) Stage {
    T u[kTile<T>][CH];
    T dt[kTile<T>][CH];
    T z[FINAL ? kTile<T> : 1][CH];
    // every number twice, as the paired operations take it
    float2 b[kTile<T>][PADDED];
    float2 c[FINAL ? kTile<T> : 1][PADDED];
};

// Two neighbouring channels of a staged row.
template <typename T>
__device__ __forceinline__ float2 load_two(const T *p)
{
    const Pack<T, 2> v = *reinterpret_cast<const Pack<T, 2> *>(p);
    return make_float2(Elem<T>::get(v.v[0]), Elem<T>::get(v.v[1]));
}

// A thread carries two neighbouring channels, each pair of registers holding
// one state of both, so that step sizes, inputs and gates are pairs as they
// come, and a staged b or c serves two channels.  G lanes share the channels'
// states, NS each.  FINAL false: the first pass, over the spans that others
// follow.  grid (items * channel blocks).
template <typename T, int NS, int G, bool WIDE, bool FINAL>
__global__ void __launch_bounds__(kScanThreads, 5) scan_kernel(ScanArgs p, Spans w)
{
    constexpr int kRows = kTile<T>;
    constexpr int kChannels = 2 * kScanThreads / G;
    constexpr int kPadded = NS * G;
    // 16 states fill all banks: their groups stand 16 bytes further apart, so
    // that the lanes of a channel read different ones
    constexpr int kGap = NS == 16 && G > 1 ? 2 : 0;
    constexpr int V = Elem<T>::kVector;
    extern __shared__ __align__(16) unsigned char shared[];
    typedef Stage<T, kChannels, kPadded + kGap * G, FINAL> StageT;
    StageT *stages = reinterpret_cast<StageT *>(shared);

    if (!FINAL)
        ptx::griddep_launch_dependents();
    const int block = blockIdx.x % w.blocks, item = blockIdx.x / w.blocks;
    int span, s;
    if (w.items) {
        ptx::griddep_wait();  // the order
        const int2 at = item < *w.count ? w.items[item] : make_int2(0, -1);
        s = at.x;
        span = at.y;
    } else if (w.each) {
        s = item / w.each;
        span = item % w.each;
    } else {
        s = tile_owner(p.seq, item, w.chunk, &span);
    }
    const int seq_begin = sequence_begin(p.seq, s), seq_end = sequence_end(p.seq, s);
    const int length = seq_end - seq_begin;
    const int spans = length > 0 ? (length - 1) / w.chunk + 1 : 1;  // (one to keep the state)
    if (span < 0 || span >= spans || (!FINAL && span == spans - 1)) {
        if (FINAL)  // what follows this kernel must not overtake the first pass
            ptx::griddep_wait();
        return;
    }
    // the sequence's first span number
    const long long first = w.each ? static_cast<long long>(s) * w.each : seq_begin / w.chunk + s;
    const bool last = span == spans - 1;  // (never in the first pass)
    const int begin = seq_begin + span * w.chunk;
    const int end = last ? seq_end : begin + w.chunk;

    const int per_group = p.channels / p.groups;
    const int blocks = (per_group + kChannels - 1) / kChannels;
    const int group = block / blocks;
    const int local0 = (block % blocks) * kChannels;
    const int here = min(kChannels, per_group - local0);  // channels of this block
    const int c0 = group * per_group + local0;
    const int ch = threadIdx.x / G * 2;
    const bool live0 = ch < here, live1 = ch + 1 < here;
    const int d0 = c0 + (live0 ? ch : 0), d1 = c0 + (live1 ? ch + 1 : 0);
    const int n0 = threadIdx.x % G * NS, n0_staged = threadIdx.x % G * (NS + kGap);
    const int slot = sequence_slot(p.slots, s);
    const bool resumes = slot >= 0 && sequence_resumes(p.slots, s);
    // whole quads where each channel's states start on a 16-byte boundary
    const bool quads = p.states == kPadded && NS % 4 == 0 &&
                       (reinterpret_cast<uintptr_t>(p.state) & 15) == 0;
    const auto kept = [&](long long at) {
        return w.states + ((at * w.blocks + block) * NS) * kScanThreads + threadIdx.x;
    };
    const auto kept_sum = [&](long long at) {
        return w.sums + (at * w.blocks + block) * kScanThreads + threadIdx.x;
    };

    Pair h[NS], a[NS];
#pragma unroll
    for (int n = 0; n < NS; ++n) {
        const int k = place_state(n0 + n, p.states);
        a[n] = make_pair(kLog2e * __ldg(p.a + static_cast<long long>(d0) * p.states + k),
                         kLog2e * __ldg(p.a + static_cast<long long>(d1) * p.states + k));
        h[n] = 0;
    }
    float *state0 = p.state + (static_cast<long long>(slot) * p.channels + d0) * p.states;
    float *state1 = p.state + (static_cast<long long>(slot) * p.channels + d1) * p.states;
    const auto start_from_state = [&]() {
        if (quads) {
#pragma unroll
            for (int n = 0; n < NS / 4 * 4; n += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(state0 + n0 + n);
                const float4 y = *reinterpret_cast<const float4 *>(state1 + n0 + n);
                h[n] = make_pair(x.x, y.x);
                h[n + 1] = make_pair(x.y, y.y);
                h[n + 2] = make_pair(x.z, y.z);
                h[n + 3] = make_pair(x.w, y.w);
            }
        } else {
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                const int k = place_state(n0 + n, p.states);
                h[n] = make_pair(state0[k], state1[k]);
            }
        }
    };
    // staging: u, dt and z as they are, asynchronously; b and c as fp32
    constexpr int kFetch = (kRows * kPadded + kScanThreads - 1) / kScanThreads;
    constexpr int kAcross = WIDE ? kChannels / V : kChannels;  // copies of a row
    const T *u = static_cast<const T *>(p.u) + c0;
    const T *dt = static_cast<const T *>(p.dt) + c0;
    const T *z = FINAL && p.z ? static_cast<const T *>(p.z) + c0 : nullptr;
    const T *b = static_cast<const T *>(p.b) + group * p.states;
    const T *c = static_cast<const T *>(p.c) + group * p.states;
    // a thread's k-th b and c: row fetch_t + row(k), place fetch_n + col(k)
    constexpr int kFetchRows = kScanThreads / kPadded;
    constexpr int kWide = kPadded / kScanThreads > 0 ? kPadded / kScanThreads : 1;
    const auto row = [](int k) { return kFetchRows ? k * kFetchRows : k / kWide; };
    const auto col = [](int k) { return kFetchRows ? 0 : k % kWide * kScanThreads; };
    const int fetch_t = threadIdx.x / kPadded, fetch_n = threadIdx.x % kPadded;
    T fetch_b[kFetch], fetch_c[kFetch];
    const auto fetch = [&](int t0, StageT &st) {
        const int count = min(kRows, end - t0);
        if constexpr (WIDE) {
            constexpr int kRowsAtOnce = kScanThreads / kAcross > 0 ? kScanThreads / kAcross : 1;
            static_assert(kAcross <= kScanThreads &&
                              (kRows % kRowsAtOnce == 0 || kRowsAtOnce > kRows),
                          "copies");
            const int t = threadIdx.x / kAcross, at = threadIdx.x % kAcross * V;
            const T *from_u = u + (t0 + t) * p.u_stride + at;
            const T *from_dt = dt + (t0 + t) * p.dt_stride + at;
            const T *from_z = z + (t0 + t) * p.z_stride + at;
#pragma unroll
            for (int i = 0; i < kRows; i += kRowsAtOnce) {
                if (t + i < count && at < here) {
                    ptx::cp_async_16(ptx::smem_u32(&st.u[t + i][at]), from_u + i * p.u_stride, 16);
                    ptx::cp_async_16(ptx::smem_u32(&st.dt[t + i][at]), from_dt + i * p.dt_stride, 16);
                    if (z)
                        ptx::cp_async_16(ptx::smem_u32(&st.z[t + i][at]), from_z + i * p.z_stride,
                                         16);
                }
            }
            ptx::cp_async_commit();
        } else {
            for (int i = threadIdx.x; i < count * kAcross; i += kScanThreads) {
                const int t = i / kAcross, at = i % kAcross;
                if (at < here) {
                    st.u[t][at] = u[(t0 + t) * p.u_stride + at];
                    st.dt[t][at] = dt[(t0 + t) * p.dt_stride + at];
                    if (z)
                        st.z[t][at] = z[(t0 + t) * p.z_stride + at];
                }
            }
        }
        const T *from_b = b + (t0 + fetch_t) * p.b_stride;
        const T *from_c = c + (t0 + fetch_t) * p.c_stride;
#pragma unroll
        for (int k = 0; k < kFetch; ++k) {
            const bool in = fetch_t + row(k) < count;
            const int n = place_state(fetch_n + col(k), p.states);
            fetch_b[k] = in ? from_b[row(k) * p.b_stride + n] : Elem<T>::put(0.0f);
            if (FINAL)
                fetch_c[k] = in ? from_c[row(k) * p.c_stride + n] : Elem<T>::put(0.0f);
        }
    };
    const auto settle = [&](StageT &st) {
#pragma unroll
        for (int k = 0; k < kFetch; ++k) {
            if (fetch_t + row(k) < kRows) {
                const int n = fetch_n + col(k), at = n + n / NS * kGap;
                const float x = Elem<T>::get(fetch_b[k]);
                st.b[fetch_t + row(k)][at] = make_float2(x, x);
                if (FINAL) {
                    const float y = place_share(n, p.states, kPadded) * Elem<T>::get(fetch_c[k]);
                    st.c[fetch_t + row(k)][at] = make_float2(y, y);
                }
            }
        }
        if (WIDE)
            ptx::cp_async_wait_all();
        __syncthreads();
    };

    int stage = 0;
    if (begin < end)
        fetch(begin, stages[0]);
    const Pair skip = p.skip ? make_pair(__ldg(p.skip + d0), __ldg(p.skip + d1)) : 0;
    const Pair dt_bias = p.dt_bias ? make_pair(__ldg(p.dt_bias + d0), __ldg(p.dt_bias + d1)) : 0;
    if (FINAL)
        ptx::griddep_wait();
    if (!FINAL && span == 0 && resumes) {
        start_from_state();
        Pair *to = kept(first + spans - 1);
#pragma unroll
        for (int n = 0; n < NS; ++n)
            to[n * kScanThreads] = h[n];
    }
    if (FINAL && spans > 1) {
        // the state that this span starts from, as carry_kernel left it
        if (span > 0 || resumes) {
            const Pair *from = kept(first + (span > 0 ? span - 1 : spans - 1));
#pragma unroll
            for (int n = 0; n < NS; ++n)
                h[n] = from[n * kScanThreads];
        }
    } else if (FINAL && resumes) {
        start_from_state();
    }

    Pair sum = 0;
    T *y = static_cast<T *>(p.y) + c0;
    // TOKENS tokens of the staged tile from its row t on
    const auto advance = [&](StageT &st, int t, auto tokens) {
        constexpr int kTokens = decltype(tokens)::value;
        Pair in[kTokens], step[kTokens], add[kTokens], out[kTokens];
#pragma unroll
        for (int j = 0; j < kTokens; ++j) {
            const float2 v = load_two(&st.u[t + j][ch]), x = load_two(&st.dt[t + j][ch]);
            in[j] = make_pair(v.x, v.y);
            step[j] = add2(make_pair(x.x, x.y), dt_bias);
            out[j] = step[j];
        }
        // (chosen, not branched: the tokens' work stays one straight line)
        softplus_pairs(out);
#pragma unroll
        for (int j = 0; j < kTokens; ++j) {
            step[j] = p.softplus ? out[j] : step[j];
            add[j] = mul2(step[j], in[j]);
            if (!FINAL)
                sum = add2(sum, step[j]);
        }
#pragma unroll
        for (int j = 0; j < kTokens; ++j) {
            Pair even = 0, odd = 0;
            if (FINAL && (G == 1 || n0 == 0))
                even = p.skip ? mul2(skip, in[j]) : 0;  // (0 times an infinity is no 0)
#pragma unroll
            for (int n = 0; n < NS; n += 2) {
                const ulonglong2 bn = *reinterpret_cast<const ulonglong2 *>(&st.b[t + j][n0_staged + n]);
                h[n] = fma2(ex2_pair(mul2(step[j], a[n])), h[n], mul2(add[j], bn.x));
                h[n + 1] = fma2(ex2_pair(mul2(step[j], a[n + 1])), h[n + 1], mul2(add[j], bn.y));
                if (FINAL) {
                    const ulonglong2 cn =
                        *reinterpret_cast<const ulonglong2 *>(&st.c[t + j][n0_staged + n]);
                    even = fma2(h[n], cn.x, even);
                    odd = fma2(h[n + 1], cn.y, odd);
                }
            }
            if (FINAL)
                out[j] = add2(even, odd);
        }
        Pair gate[kTokens];
#pragma unroll
        for (int j = 0; FINAL && j < kTokens; ++j) {
#pragma unroll
            for (int m = 1; m < G; m <<= 1) {
                const float2 v = split_pair(out[j]);
                out[j] = add2(out[j], make_pair(__shfl_xor_sync(0xffffffffu, v.x, m),
                                                __shfl_xor_sync(0xffffffffu, v.y, m)));
            }
            const float2 g = load_two(&st.z[t + j][ch]);
            gate[j] = make_pair(g.x, g.y);
        }
        if (FINAL)
            silu_pairs(gate);
#pragma unroll
        for (int j = 0; FINAL && j < kTokens; ++j) {
            const Pair gated = mul2(out[j], gate[j]);
            const float2 v = split_pair(z ? gated : out[j]);
            // the output takes the place of the token's gate (of a channel's
            // lanes only the first one's output counts)
            Pack<T, 2> q;
            q.v[0] = Elem<T>::put(v.x);
            q.v[1] = Elem<T>::put(v.y);
            if (G == 1 || n0 == 0)
                *reinterpret_cast<Pack<T, 2> *>(&st.z[t + j][ch]) = q;
        }
    };
    // the outputs of the tile at t0, by the threads that fetched their places
    // and fetch into them again
    const auto flush = [&](int t0, const StageT &st) {
        const int count = min(kRows, end - t0);
        if constexpr (WIDE) {
            constexpr int kRowsAtOnce = kScanThreads / kAcross > 0 ? kScanThreads / kAcross : 1;
            const int t = threadIdx.x / kAcross, at = threadIdx.x % kAcross * V;
            T *to = y + (t0 + t) * p.y_stride + at;
#pragma unroll
            for (int i = 0; i < kRows; i += kRowsAtOnce)
                if (t + i < count && at < here)
                    *reinterpret_cast<uint4 *>(to + i * p.y_stride) =
                        *reinterpret_cast<const uint4 *>(&st.z[t + i][at]);
        } else {
            for (int i = threadIdx.x; i < count * kAcross; i += kScanThreads) {
                const int t = i / kAcross, at = i % kAcross;
                if (at < here)
                    y[(t0 + t) * p.y_stride + at] = st.z[t][at];
            }
        }
    };
    for (int t0 = begin; t0 < end; t0 += kRows) {
        StageT &st = stages[stage];
        settle(st);
        stage ^= 1;
        if (FINAL && t0 > begin)
            flush(t0 - kRows, stages[stage]);
        if (t0 + kRows < end)
            fetch(t0 + kRows, stages[stage]);
        const int count = min(kRows, end - t0);
        int t = 0;
#pragma unroll 1
        for (; t + kStep <= count; t += kStep)
            advance(st, t, std::integral_constant<int, kStep>());
#pragma unroll 1
        for (; t < count; ++t)
            advance(st, t, std::integral_constant<int, 1>());
    }
    if (FINAL && begin < end) {
        __syncthreads();
        flush(begin + (end - begin - 1) / kRows * kRows, stages[stage ^ 1]);
    }
    if (!FINAL) {
        Pair *to = kept(first + span);
#pragma unroll
        for (int n = 0; n < NS; ++n)
            to[n * kScanThreads] = h[n];
        *kept_sum(first + span) = sum;
    } else if (last && slot >= 0) {
        if (quads) {
#pragma unroll
            for (int n = 0; n < NS / 4 * 4; n += 4) {
                const float2 v0 = split_pair(h[n]), v1 = split_pair(h[n + 1]),
                             v2 = split_pair(h[n + 2]), v3 = split_pair(h[n + 3]);
                if (live0)
                    *reinterpret_cast<float4 *>(state0 + n0 + n) =
                        make_float4(v0.x, v1.x, v2.x, v3.x);
                if (live1)
                    *reinterpret_cast<float4 *>(state1 + n0 + n) =
                        make_float4(v0.y, v1.y, v2.y, v3.y);
            }
        } else {
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                const float2 v = split_pair(h[n]);
                if (n0 + n < p.states) {
                    if (live0)
                        state0[n0 + n] = v.x;
                    if (live1)
                        state1[n0 + n] = v.y;
                }
            }
        }
    }
}

// Between the passes: turns what the first pass left of each span into the
// state after it, every span carrying the state before it on by
// e^(a * its step sizes' sum).  Token by token an infinite state stays infinite
// however far it decays, so it is not multiplied by a product that has become 0
// on the way (by one of an infinite step size it is).  A thread follows one state of a channel pair
// over a sequence's spans, loading kCarry of them together.  grid (sequences *
// channel blocks * NS).
constexpr int kCarry = 16;
template <int NS, int G>
__global__ void __launch_bounds__(kScanThreads) carry_kernel(ScanArgs p, Spans w)
{
    ptx::griddep_launch_dependents();
    const int n = blockIdx.x % NS, block = blockIdx.x / NS % w.blocks;
    const int s = blockIdx.x / NS / w.blocks;
    const int begin = sequence_begin(p.seq, s), length = sequence_end(p.seq, s) - begin;
    const int spans = length > 0 ? (length - 1) / w.chunk + 1 : 1;
    const int left = spans - 1;  // spans that left something; the first is complete
    const long long first = w.each ? static_cast<long long>(s) * w.each : begin / w.chunk + s;
    const int per_group = p.channels / p.groups, channels = 2 * kScanThreads / G;
    const int blocks = (per_group + channels - 1) / channels;
    const int local = (block % blocks) * channels + threadIdx.x / G * 2;
    const int d = block / blocks * per_group + local;
    const int k0 = place_state(threadIdx.x % G * NS + n, p.states);
    const auto decay = [&](int c) {
        return local + c < per_group
                   ? kLog2e * __ldg(p.a + static_cast<long long>(d + c) * p.states + k0)
                   : 0.0f;
    };
    const Pair a = left > 1 ? make_pair(decay(0), decay(1)) : 0;
    ptx::griddep_wait();
    if (left <= 1)
        return;
    const long long row = static_cast<long long>(w.blocks) * kScanThreads;  // pairs of a span's sums
    Pair *state = w.states + (first * w.blocks + block) * NS * kScanThreads + n * kScanThreads +
                  threadIdx.x;
    const Pair *sum = w.sums + (first * w.blocks + block) * kScanThreads + threadIdx.x;
    Pair h = state[0];
    for (int k = 1; k < left; k += kCarry) {
        Pair ends[kCarry], sums[kCarry];
#pragma unroll
        for (int j = 0; j < kCarry; ++j)
            if (k + j < left) {
                ends[j] = state[(k + j) * row * NS];
                sums[j] = sum[(k + j) * row];
            }
#pragma unroll
        for (int j = 0; j < kCarry; ++j)
            if (k + j < left) {
                const float2 far = split_pair(mul2(sums[j], a)), from = split_pair(h);
                const float2 by = split_pair(ex2_pair(make_pair(far.x, far.y)));
                const bool x_stays = isinf(from.x) && far.x > -INFINITY;
                const bool y_stays = isinf(from.y) && far.y > -INFINITY;
                h = fma2(make_pair(x_stays ? 1.0f : by.x, y_stays ? 1.0f : by.y), h, ends[j]);
                state[(k + j) * row * NS] = h;
            }
    }
}

template <typename T, int NS, int G, bool WIDE>
int launch_prompts(const ScanArgs &p, const Plan &plan, void *workspace, cudaStream_t stream)
{
    constexpr int kChannels = 2 * kScanThreads / G;
    if (plan.spans * plan.blocks > 0x7fffffffll ||
        (plan.whole > 0 && plan.blocks * p.seq.count * NS > 0x7fffffffll))  // carry_kernel's grid
        return fail(LSTM_E_OVERFLOW, "lstm_selective_scan: %d sequences, %d tokens, %d channels",
                    p.seq.count, p.seq.tokens, p.channels);
    Spans w = {plan.chunk, plan.each, nullptr, nullptr, static_cast<int>(plan.blocks),
               static_cast<Pair *>(workspace), nullptr};
    Pair *end = w.states;
    if (plan.whole > 0) {
        w.sums = w.states + plan.spans * plan.blocks * kScanThreads * NS;
        end = w.sums + plan.spans * plan.blocks * kScanThreads;
    }
    constexpr size_t kShared = 2 * sizeof(Stage<T, kChannels, (NS + (NS == 16 && G > 1 ? 2 : 0)) * G, true>);
    constexpr size_t kSharedFirst = 2 * sizeof(Stage<T, kChannels, (NS + (NS == 16 && G > 1 ? 2 : 0)) * G, false>);
    static SharedMemory allowed, allowed_first;
    int st;
    if ((st = allowed.allow(scan_kernel<T, NS, G, WIDE, true>, kShared)) ||
        (st = allowed_first.allow(scan_kernel<T, NS, G, WIDE, false>, kSharedFirst)))
        return st;
    // each kernel may start while the one before it ends; it waits for it
    // before it reads what that left
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = attr;
    if (plan.order) {
        int2 *items = reinterpret_cast<int2 *>(end);
        int *count = reinterpret_cast<int *>(items + plan.spans);
        if ((st = launch_order(p.seq, plan.chunk, static_cast<int>(plan.spans), items, count,
                               stream)))
            return st;
        w.items = items;
        w.count = count;
        cfg.numAttrs = 1;
    }
    cfg.blockDim = dim3(kScanThreads);
    if (plan.whole > 0) {
        if ((st = check_launch_injection("lstm_selective_scan")))
            return st;
        // (in order, the spans that others follow come first)
        cfg.gridDim = dim3(static_cast<unsigned>((plan.order ? plan.whole : plan.spans) * plan.blocks));
        cfg.dynamicSmemBytes = kSharedFirst;
        if ((st = cuda_status(cudaLaunchKernelEx(&cfg, scan_kernel<T, NS, G, WIDE, false>, p, w),
                              "lstm_selective_scan launch")))
            return st;
        cfg.numAttrs = 1;
        if ((st = check_launch_injection("lstm_selective_scan")))
            return st;
        cfg.gridDim = dim3(static_cast<unsigned>(p.seq.count * plan.blocks * NS));
        cfg.dynamicSmemBytes = 0;
        if ((st = cuda_status(cudaLaunchKernelEx(&cfg, carry_kernel<NS, G>, p, w),
                              "lstm_selective_scan launch")))
            return st;
    }
    if ((st = check_launch_injection("lstm_selective_scan")))
        return st;
    cfg.gridDim = dim3(static_cast<unsigned>(plan.spans * plan.blocks));
    cfg.dynamicSmemBytes = kShared;
    return cuda_status(cudaLaunchKernelEx(&cfg, scan_kernel<T, NS, G, WIDE, true>, p, w),
                       "lstm_selective_scan launch");
}

template <typename T, int NS, int G>
int launch_aligned(const ScanArgs &p, const Plan &plan, void *workspace, cudaStream_t stream)
{
    constexpr int V = Elem<T>::kVector;
    const int size = sizeof(T);
    // 16-byte copies where every row of u, dt, z and y, and every group of
    // channels, starts on a 16-byte boundary
    const bool wide = p.channels / p.groups % V == 0 && rows_aligned(p.u, p.u_stride, size) &&
                      rows_aligned(p.dt, p.dt_stride, size) &&
                      rows_aligned(p.y, p.y_stride, size) &&
                      (!p.z || rows_aligned(p.z, p.z_stride, size));
    return wide ? launch_prompts<T, NS, G, true>(p, plan, workspace, stream)
                : launch_prompts<T, NS, G, false>(p, plan, workspace, stream);
}

template <typename T>
int launch_scan(const ScanArgs &p, const Plan &plan, void *workspace, cudaStream_t stream)
{
    switch (plan.states * 16 + plan.lanes) {
    case 4 * 16 + 1:
        return launch_aligned<T, 4, 1>(p, plan, workspace, stream);
    case 4 * 16 + 2:
        return launch_aligned<T, 4, 2>(p, plan, workspace, stream);
    case 4 * 16 + 4:
        return launch_aligned<T, 4, 4>(p, plan, workspace, stream);
    case 8 * 16 + 1:
        return launch_aligned<T, 8, 1>(p, plan, workspace, stream);
    case 8 * 16 + 2:
        return launch_aligned<T, 8, 2>(p, plan, workspace, stream);
    case 16 * 16 + 1:
        return launch_aligned<T, 16, 1>(p, plan, workspace, stream);
    case 16 * 16 + 2:
        return launch_aligned<T, 16, 2>(p, plan, workspace, stream);
    case 16 * 16 + 4:
        return launch_aligned<T, 16, 4>(p, plan, workspace, stream);
    default:
        return launch_aligned<T, 16, 8>(p, plan, workspace, stream);
    }
}

}  // namespace
}  // namespace lstm
