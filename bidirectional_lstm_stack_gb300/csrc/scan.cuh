// What the selective scan's translation units share: its arguments, how a
// call's prompts are divided, and the paired arithmetic.
//
//   h[n] = e^(s a[n]) h[n] + s u b[t][n],   v = sum_n h[n] c[t][n] + skip u
//
// per channel, with s the step size of that token and channel and the states
// h in fp32 registers from the first token to the last.
#pragma once

#include "ops.cuh"

namespace lstm {

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

// The first pass and the second one over spans of `chunk` tokens (chunk tiles,
// in tile_owner's numbering).  The first pass leaves, per span, channel and
// state, the state after the span when it starts from zeros (the sequence's
// first span: from its own start), and per span and channel the sum of the
// span's step sizes; carry_kernel joins them into the state that each span
// starts from.  A sequence's last span has nothing to leave; its place
// holds the state that the sequence starts from, which the second pass may
// not read where it is kept, because the last span replaces it.
//
// Work items are spans.  Sequences of equal length have `each` spans each, in
// order.  Of unequal ones an order is made on the GPU (order_kernel) when
// there is much work: whole spans first, then the sequences' last spans from
// the longest to the shortest, so that the last blocks to start are short
// ones; else an item is a span number.
struct Spans {
    int chunk;
    int each;           // 0: unequal lengths
    const int2 *items;  // (sequence, span) in order, or null
    const int *count;   // of items
    int blocks;         // channel blocks of a group * groups
    Pair *states;  // [numbers][channel blocks][states of a thread][threads]
    Pair *sums;    // [numbers][channel blocks][threads]
};

constexpr int kMostChannels = 1 << 30;  // and numbers of a row of b or c
constexpr int kScanThreads = 64;  // of a block; with two channels a thread

// How a call's prompts are worked on: the same for its workspace's size and
// for its launches.
struct Plan {
    int states;        // a thread's
    int lanes;         // a pair of channels'
    long long blocks;  // channel blocks
    int chunk;         // tokens of a span
    long long spans;   // at most so many
    long long whole;   // spans that others follow: at most so many
    int each;          // spans of a sequence, where all have the same length
    bool order;        // whether order_kernel runs
    size_t bytes;      // of workspace: states, sums, items, count
};

// The prompts' kernels, one translation unit a type.
int launch_scan_f32(const ScanArgs &p, const Plan &plan, void *workspace, cudaStream_t stream);
int launch_scan_bf16(const ScanArgs &p, const Plan &plan, void *workspace, cudaStream_t stream);
int launch_scan_f16(const ScanArgs &p, const Plan &plan, void *workspace, cudaStream_t stream);
// Puts the spans of sequences of unequal lengths in order (scan.cu).
int launch_order(const Sequences &q, int chunk, int limit, int2 *items, int *count,
                 cudaStream_t stream);
// The single tokens' kernel (scan_step.cu).
int launch_scan_step(const ScanArgs &p, int dtype, cudaStream_t stream);

#ifdef __CUDACC__

// The prompts' lanes have places for a power of two of states, at most twice as
// many as there are (four for a single one).  The places beyond the last state
// hold the first ones again, and a state's output is shared out evenly among its
// places, by halves (quarters), which is exact.  (Zeros in them would be NaN after
// an infinite input.)  The state of place n:
__device__ __forceinline__ int place_state(int n, int states)
{
    return n < states ? n : states > 1 ? n - states : 0;
}
// 1 / the number of places of place n's state, of `places` in all.
__device__ __forceinline__ float place_share(int n, int states, int places)
{
    return states == 1 ? 1.0f / places : place_state(n, states) + states < places ? 0.5f : 1.0f;
}

// log(1 + e^v) = max(v, 0) + log(1 + e), e = e^-|v| in (0, 1], and
// log(1 + e) = e q(e) with q of degree 8, fitted by least squares whose
// weights are moved to where the relative error is largest (Lawson's method)
// until it is level: 3e-8, and 1.7e-7 with fp32's roundings, for small e as
// for large.  (As written, the sum 1 + e would lose the small ones.)
// In place for K pairs, side by side, so that none waits for its own result.
template <int K>
__device__ __forceinline__ void softplus_pairs(Pair (&v)[K])
{
    const float c[] = {0.005232679657638073f, -0.029505178332328796f, 0.07822585105895996f,
                       -0.13663236796855927f, 0.19106002151966095f,   -0.2484298050403595f,
                       0.3331909775733948f,   -0.4999949336051941f,   0.9999999403953552f};
    Pair e[K], q[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const float2 x = split_pair(v[k]);
        e[k] = make_pair(-kLog2e * fabsf(x.x), -kLog2e * fabsf(x.y));
        v[k] = make_pair(fmaxf(x.x, 0.0f), fmaxf(x.y, 0.0f));
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
        e[k] = ex2_pair(e[k]);
#pragma unroll
    for (int k = 0; k < K; ++k)
        q[k] = fma2(e[k], make_pair(c[0], c[0]), make_pair(c[1], c[1]));
#pragma unroll
    for (int i = 2; i < 9; ++i)
#pragma unroll
        for (int k = 0; k < K; ++k)
            q[k] = fma2(q[k], e[k], make_pair(c[i], c[i]));
#pragma unroll
    for (int k = 0; k < K; ++k)
        v[k] = fma2(q[k], e[k], v[k]);
}
#endif  // __CUDACC__

}  // namespace lstm
