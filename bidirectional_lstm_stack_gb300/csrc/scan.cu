// The selective scan's entry points, and how a call's prompts are divided.
#include <math.h>

#include "scan.cuh"

namespace lstm {
namespace {

// Puts the spans of sequences of unequal lengths in order: whole spans first,
// then the last spans from long to short (by sixty-fourths of a span; within
// one, in any order: it changes no result).  One block.
constexpr int kOrderThreads = 256;
constexpr int kOrderBins = 66;  // bin 0: whole spans
__global__ void __launch_bounds__(kOrderThreads) order_kernel(Sequences q, int chunk, int2 *items,
                                                              int *count, int limit)
{
    ptx::griddep_launch_dependents();
    __shared__ int bins[kOrderBins];
    for (int i = threadIdx.x; i < kOrderBins; i += kOrderThreads)
        bins[i] = 0;
    __syncthreads();
    const auto spans_of = [&](int s, int *bin) {
        const int length = sequence_end(q, s) - sequence_begin(q, s);
        const int spans = length > 0 ? (length - 1) / chunk + 1 : 1;
        const int rest = length - (spans - 1) * chunk;  // 0 .. chunk
        *bin = 65 - static_cast<int>(64ll * rest / chunk);
        return spans;
    };
    for (int s = threadIdx.x; s < q.count; s += kOrderThreads) {
        int bin;
        const int spans = spans_of(s, &bin);
        if (spans > 1)
            atomicAdd(&bins[0], spans - 1);
        atomicAdd(&bins[bin], 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int sum = 0;
        for (int i = 0; i < kOrderBins; ++i) {
            const int n = bins[i];
            bins[i] = sum;
            sum += n;
        }
        *count = min(sum, limit);
    }
    __syncthreads();
    for (int s = threadIdx.x; s < q.count; s += kOrderThreads) {
        int bin;
        const int spans = spans_of(s, &bin);
        if (spans > 1) {
            const int at = atomicAdd(&bins[0], spans - 1);
            for (int k = 0; k < spans - 1 && at + k < limit; ++k)
                items[at + k] = make_int2(s, k);
        }
        const int at = atomicAdd(&bins[bin], 1);
        if (at < limit)  // (always, where offsets do not decrease)
            items[at] = make_int2(s, spans - 1);
    }
}

// What a plan costs, measured: a warp alone takes token_ns a token, which
// bounds the longest span, and a block of a full machine cta_ns a token, which
// bounds all of them together.  Fewer states a thread and more lanes a channel
// shorten the first and, because the lanes repeat what a channel needs once,
// lengthen the second.
struct Rate {
    int states;
    double token_ns;
    double cta_ns;
    double uneven;  // times cta_ns, where unequal lengths load the SMs unevenly
};
constexpr Rate kRates[] = {{16, 175, 0.59, 1.45}, {8, 126, 0.39, 1.0}, {4, 100, 0.26, 1.0}};
// Splitting takes two passes (the first one costs some two thirds of the
// second) and two launches more.
constexpr double kPasses = 1.7, kLaunchesNs = 5000;
constexpr int kLeastChunk = 32;

Plan make_plan(int tokens, int channels, int states, int groups, int sequences, bool equal)
{
    // The longest sequence: known, or guessed at three times the mean, as the host
    // does not see the lengths (prompts whose lengths spread evenly over a factor of
    // thirty reach 3.5 times).  Where one is much longer the guess keeps it whole:
    // 4096 tokens beside 63 prompts of one, 2048 channels x 16 states, take 479 us,
    // the 4096 alone, in spans, 80.
    const double mean = sequences > 0 ? static_cast<double>(tokens) / sequences : 0;
    const double longest = equal || sequences <= 1 ? mean : fmin(3 * mean, tokens);
    Plan best = {};
    double best_ns = 0;
    for (const Rate &rate : kRates) {
        Plan r = {};
        r.states = rate.states;
        r.lanes = 1;
        while (r.states * r.lanes < states)
            r.lanes *= 2;
        // no more than half of the places unused (place_state relies on it), and
        // at most 4 lanes of fewer than 16 states (16 of 4 would leave no channels
        // to a block)
        if (r.states >= 2 * states && r.states > 4)
            continue;
        if (r.lanes > 4 && r.states < 16)
            continue;
        if (r.lanes > 1 && r.states < 16 && states > 16)
            continue;
        const int block = 2 * kScanThreads / r.lanes;  // channels
        r.blocks = static_cast<long long>((channels / groups + block - 1) / block) * groups;
        const double work = static_cast<double>(tokens) * r.blocks;
        const double uneven = equal || sequences <= 1 ? 1.0 : rate.uneven;
        for (int split = 0; split < 2; ++split) {
            // spans that fill the machine six blocks deep (or a little less: their
            // length is rounded up to 16 tokens, so 4096 tokens of 2048 channels make
            // 52 spans of 80 in 16 channel blocks, 5.5 blocks an SM)
            long long chunk = static_cast<long long>(work / (152 * 6));
            chunk = (chunk + 15) / 16 * 16;
            if (chunk < kLeastChunk)
                chunk = kLeastChunk;
            if (split && chunk >= (equal ? longest : tokens))
                continue;
            const double ns =
                split ? kPasses * fmax(chunk * rate.token_ns, work * rate.cta_ns) + kLaunchesNs
                      : fmax(longest * rate.token_ns, work * rate.cta_ns * uneven);
            if (best_ns > 0 && ns >= best_ns)
                continue;
            best_ns = ns;
            best = r;
            // whole sequences: spans longer than all tokens together number just them
            best.chunk = split ? static_cast<int>(chunk) : tokens + 1;
        }
    }
    Plan r = best;
    const bool split = r.chunk <= tokens;
    if (equal) {
        const int length = sequences > 0 ? tokens / sequences : 0;
        r.each = split ? (length + r.chunk - 1) / r.chunk : 1;
        r.spans = static_cast<long long>(r.each) * sequences;
        r.whole = r.spans - sequences;
    } else {
        r.spans = split ? tiles_bound(tokens, sequences, r.chunk) : sequences;
        r.whole = split ? tokens / r.chunk : 0;
        r.order = sequences > 1 && r.spans * r.blocks > 152 * 2;
    }
    if (r.whole > 0)
        r.bytes = static_cast<size_t>(r.spans) * r.blocks * kScanThreads * (r.states + 1) *
                  sizeof(Pair);
    if (r.order)
        r.bytes += (r.spans + 1) * sizeof(int2);
    return r;
}

}  // namespace

int launch_order(const Sequences &q, int chunk, int limit, int2 *items, int *count,
                 cudaStream_t stream)
{
    const int st = check_launch_injection("lstm_selective_scan");
    if (st != LSTM_OK)
        return st;
    order_kernel<<<1, kOrderThreads, 0, stream>>>(q, chunk, items, count, limit);
    return cuda_status(cudaGetLastError(), "lstm_selective_scan launch");
}

namespace {

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
    // (the kernels count channels a block beyond the last and a row's b in 32 bits)
    if (p.channels > kMostChannels || wide > kMostChannels)
        return fail(LSTM_E_OVERFLOW, "%s: %d channels, %d groups of %d states (rows of at most %d)",
                    what, p.channels, p.groups, p.states, kMostChannels);
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
        plan = make_plan(rows, p.channels, p.states, p.groups, p.seq.count, !p.seq.offsets);
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
    cudaStream_t on = static_cast<cudaStream_t>(stream);
    if (step)
        return launch_scan_step(p, dtype, on);
    return dtype == LSTM_F32    ? launch_scan_f32(p, plan, workspace, on)
           : dtype == LSTM_BF16 ? launch_scan_bf16(p, plan, workspace, on)
                                : launch_scan_f16(p, plan, workspace, on);
}

}  // namespace
}  // namespace lstm

using namespace lstm;

extern "C" size_t lstm_selective_scan_workspace(int tokens, int channels, int states, int groups,
                                                int sequences, int equal_lengths)
{
    if (tokens < 0 || channels <= 0 || channels > kMostChannels || states <= 0 ||
        states > LSTM_SCAN_MAX_STATES || groups <= 0 || sequences <= 0 || tokens > kMostTokens || sequences > kMostSequences)
        return 0;
    return make_plan(tokens, channels, states, groups, sequences, equal_lengths != 0).bytes;
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
    const int st = check_sequences("lstm_selective_scan_step", sequences, sequences, nullptr);
    if (st != LSTM_OK)
        return st;
    ScanArgs p = {u, u_stride, dt, dt_stride, a, b, b_stride, c, c_stride, skip, z, z_stride,
                  dt_bias, softplus != 0, channels, states, groups, state,
                  {nullptr, sequences, 1, sequences}, {slots, nullptr, state_slots}, y, y_stride};
    return scan("lstm_selective_scan_step", p, dtype, sequences, true, nullptr, 0, stream);
}
