// Log probabilities of given tokens, the entropy and the top alternatives of
// rows of logits, in one pass over the logits.
//
// A row's softmax is summed while it streams by: with m the largest logit so
// far, s = sum e^(x - m) and w = sum e^(x - m) (x - m) are scaled by e^(m - m')
// whenever m grows to m', and at the end
//   l[v] = (x[v] - m) - ln s,   entropy = ln s - w / s.
// The top alternatives are kept as 64-bit keys, the logit's order above the
// index's, so that equal logits rank by index and no order of work changes
// the result: lane i of a warp holds the warp's i-th largest key, candidates
// above the k-th of them are collected in shared memory and merged 32 at a
// time by bitonic networks, and the warps' lists are merged at the end.
#include <cmath>

#include "ops.cuh"

namespace lstm {
namespace {

struct LogprobArgs {
    const void *logits;
    long long stride;
    const long long *tokens;
    float *logp;
    float *entropy;
    int top;
    float *top_logp;
    long long *top_ids;
    int rows;
    int vocab;
};

typedef unsigned long long Key;  // 0: below every logit's

// Increasing in the logit (NaN on top, -0 as 0), then decreasing in the index.
__device__ __forceinline__ Key make_key(float v, int index)
{
    unsigned u = __float_as_uint(v + 0.0f);
    u = isnan(v) ? 0xffffffffu : u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
    return static_cast<Key>(u) << 32 | ~static_cast<unsigned>(index);
}
__device__ __forceinline__ int key_index(Key k) { return ~static_cast<unsigned>(k); }
__device__ __forceinline__ float key_value(Key k)
{
    const unsigned u = static_cast<unsigned>(k >> 32);
    return __uint_as_float(u >> 31 ? u ^ 0x80000000u : ~u);
}

// The larger, or NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

struct Stats {
    float m;  // the largest logit
    float s;  // sum e^(x - m)
    float w;  // sum e^(x - m) (x - m)
};
constexpr float kInf = INFINITY;

__device__ __forceinline__ Stats rescale(Stats a, float m)
{
    const float f = ex2((a.m - m) * kLog2e);
    // nothing summed, or nothing left of it: also where a.m - m is infinite
    if (a.s == 0.0f || f == 0.0f)
        return {m, 0.0f, 0.0f};
    return {m, a.s * f, (a.w + a.s * (a.m - m)) * f};
}
__device__ __forceinline__ Stats join(Stats a, Stats b)
{
    const float m = max_nan(a.m, b.m);
    a = rescale(a, m);
    b = rescale(b, m);
    return {m, a.s + b.s, a.w + b.w};
}
template <int LANES>
__device__ __forceinline__ Stats lanes_join(Stats a)
{
#pragma unroll
    for (int i = LANES / 2; i; i >>= 1) {
        const Stats b = {__shfl_xor_sync(0xffffffffu, a.m, i), __shfl_xor_sync(0xffffffffu, a.s, i),
                         __shfl_xor_sync(0xffffffffu, a.w, i)};
        a = join(a, b);
    }
    return a;
}

// One compare-exchange of a bitonic network: lane i with lane i ^ step, the
// larger key to the lane whose `upper` is set.
__device__ __forceinline__ Key exchange(Key k, int step, bool upper)
{
    const Key other = __shfl_xor_sync(0xffffffffu, k, step);
    return (k > other) == upper ? k : other;
}
// Sorts the keys of LANES consecutive lanes, largest in lane 0 (or, ASCENDING,
// smallest).
template <int LANES, bool ASCENDING>
__device__ __forceinline__ Key lanes_sort(Key k)
{
    const int lane = threadIdx.x % LANES;
#pragma unroll
    for (int size = 2; size <= LANES; size <<= 1)
#pragma unroll
        for (int step = size / 2; step; step >>= 1)
            k = exchange(k, step,
                         (((lane & step) == 0) == ((lane & size) == 0)) != ASCENDING);
    return k;
}
// The 32 largest of a warp's sorted list and 32 other keys in ascending order.
__device__ __forceinline__ Key warp_merge(Key list, Key ascending)
{
    Key k = list > ascending ? list : ascending;  // bitonic
#pragma unroll
    for (int step = 16; step; step >>= 1)
        k = exchange(k, step, (threadIdx.x & step) == 0);
    return k;
}

__device__ __forceinline__ void write_stats(const LogprobArgs &p, int row, const Stats &a,
                                            const float ln_s, float token_logit)
{
    const bool empty = a.s == 0.0f;
    if (p.logp) {
        const long long token = p.tokens[row];
        float v = (token_logit - a.m) - ln_s;
        if (empty)
            v = -kInf;
        if (token < 0)
            v = 0.0f;
        else if (token >= p.vocab)
            v = NAN;
        p.logp[row] = v;
    }
    if (p.entropy)
        p.entropy[row] = empty ? 0.0f : ln_s - a.w / a.s;
}
__device__ __forceinline__ void write_top(const LogprobArgs &p, int row, int i, Key k,
                                          const Stats &a, const float ln_s)
{
    const long long at = static_cast<long long>(row) * p.top + i;
    p.top_ids[at] = key_index(k);
    p.top_logp[at] = a.s == 0.0f ? -kInf : (key_value(k) - a.m) - ln_s;
}
template <typename T>
__device__ __forceinline__ float token_logit(const LogprobArgs &p, const T *x, int row)
{
    if (!p.logp)
        return 0.0f;
    const long long token = p.tokens[row];
    return token >= 0 && token < p.vocab ? Elem<T>::get(x[token]) : 0.0f;
}

// ---- rows of at most 32 logits: LANES lanes a row -------------------------------
constexpr int kSmallThreads = 128;

template <typename T, int LANES>
__global__ void __launch_bounds__(kSmallThreads) small_kernel(LogprobArgs p)
{
    const long long row0 =
        (static_cast<long long>(blockIdx.x) * kSmallThreads + threadIdx.x) / LANES;
    const bool live = row0 < p.rows;
    const int row = live ? static_cast<int>(row0) : 0;
    const int i = threadIdx.x % LANES;
    const T *x = static_cast<const T *>(p.logits) + row * p.stride;
    const float v = i < p.vocab ? Elem<T>::get(x[i]) : -kInf;
    float m = v;
#pragma unroll
    for (int k = LANES / 2; k; k >>= 1)
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, k));
    const float d = v - (m == -kInf ? 0.0f : m);
    const float e = ex2(d * kLog2e);
    Stats a = {m, e, e * fmaxf(d, -1e30f)};
#pragma unroll
    for (int k = LANES / 2; k; k >>= 1) {
        a.s += __shfl_xor_sync(0xffffffffu, a.s, k);
        a.w += __shfl_xor_sync(0xffffffffu, a.w, k);
    }
    const float ln_s = logf(a.s);
    const float given = token_logit(p, x, row);
    if (live && i == 0)
        write_stats(p, row, a, ln_s, given);
    if (p.top) {
        const Key k = lanes_sort<LANES, false>(i < p.vocab ? make_key(v, i) : 0);
        if (live && i < p.top)
            write_top(p, row, i, k, a, ln_s);
    }
}

// ---- longer rows: WARPS warps of each of a cluster's blocks a row ----------------
// A thread's batch: kBatch 16-byte vectors, loaded together.
constexpr int kBatch = 4;
constexpr int kMaxCluster = 8;

// A warp's running top list and its candidates.
struct TopList {
    Key list;       // lane i: the i-th largest so far
    Key bar;        // only keys above it matter
    float bar_value;
    int waiting;    // candidates in the buffer, fewer than 32 between calls
    Key *buffer;    // 64 keys of shared memory

    __device__ __forceinline__ void raise(int top)
    {
        const Key k = __shfl_sync(0xffffffffu, list, top - 1);
        bar = k > bar ? k : bar;
        bar_value = bar ? key_value(bar) : -kInf;
    }
    __device__ __forceinline__ void add(bool yes, Key k, int top)
    {
        const unsigned mask = __ballot_sync(0xffffffffu, yes);
        if (!mask)
            return;
        const int lane = threadIdx.x % 32;
        if (yes)
            buffer[waiting + __popc(mask & ((1u << lane) - 1))] = k;
        waiting += __popc(mask);
        __syncwarp();
        if (waiting < 32)
            return;
        const Key first = buffer[lane], rest = buffer[32 + lane];
        __syncwarp();
        buffer[lane] = rest;
        waiting -= 32;
        __syncwarp();
        list = warp_merge(list, lanes_sort<32, true>(first));
        raise(top);
    }
    __device__ __forceinline__ void finish()
    {
        const int lane = threadIdx.x % 32;
        const Key k = lane < waiting ? buffer[lane] : 0;
        list = warp_merge(list, lanes_sort<32, true>(k));
    }
};

__device__ __forceinline__ void store_cluster(uint32_t addr, unsigned long long v)
{
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

template <typename T, int WARPS, bool TOP>
__global__ void __launch_bounds__(WARPS * 32) row_kernel(LogprobArgs p)
{
    constexpr int V = Elem<T>::kVector;
    constexpr int kThreads = WARPS * 32;
    __shared__ Key buffers[TOP ? WARPS : 1][64];
    __shared__ Key lists[TOP ? WARPS : 1][32];
    __shared__ Stats stats[WARPS];
    // what the cluster's other blocks send to its first
    __shared__ Key block_lists[TOP ? kMaxCluster : 1][32];
    __shared__ __align__(16) float block_stats[kMaxCluster][4];
    const uint32_t rank = ptx::cluster_ctarank();
    const int blocks = gridDim.y;  // the cluster's
    const int row = blockIdx.x;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    if (blocks > 1)
        ptx::cluster_arrive_release();
    const T *x = static_cast<const T *>(p.logits) + row * p.stride;
    const float given = threadIdx.x == 0 && rank == 0 ? token_logit(p, x, row) : 0.0f;
    // the row in 16-byte vectors of its own alignment: vector q holds the
    // elements q * V - shift .. + V-1, the first and the last partly outside
    const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    const int vectors = static_cast<int>((static_cast<long long>(p.vocab) + shift + V - 1) / V);
    const int share = (vectors + blocks - 1) / blocks;
    const int first = min(vectors, static_cast<int>(rank) * share);
    const int last = min(vectors, first + share);

    Stats a = {-kInf, 0.0f, 0.0f};
    TopList top = {0, 0, -kInf, 0, buffers[TOP ? warp : 0]};
    // the same number of turns for all lanes of a warp
    for (int q0 = first + warp * 32; q0 < last; q0 += kBatch * kThreads) {
        float v[kBatch][V];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int q = q0 + j * kThreads + lane;
            const int e0 = q * V - shift;
            if (q < last && e0 >= 0 && e0 + V <= p.vocab) {
                unpack<T, V>(load_pack<T, V>(x + e0), v[j]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    v[j][i] = q < last && e0 + i >= 0 && e0 + i < p.vocab ? Elem<T>::get(x[e0 + i])
                                                                         : -kInf;
            }
        }
        float most = v[0][0];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i)
                most = max_nan(most, v[j][i]);
        const float m = max_nan(a.m, most);
        if (!(m == a.m))
            a = rescale(a, m);
        const float base = m == -kInf ? 0.0f : m;
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = v[j][i] - base;
                const float e = ex2(d * kLog2e);
                a.s += e;
                a.w = fmaf(e, fmaxf(d, -1e30f), a.w);
            }
        if (TOP) {
            if (top.bar == 0) {
                // a first bar: the lanes' largest are `top` different logits
                // (as keys of an index above the batch's, which rank below their own)
                const Key k = lanes_sort<32, false>(
                    most == -kInf ? 0 : make_key(most, (q0 + kBatch * kThreads) * V));
                top.bar = __shfl_sync(0xffffffffu, k, p.top - 1);
                top.bar_value = top.bar ? key_value(top.bar) : -kInf;
            }
            if (__any_sync(0xffffffffu, !(most < top.bar_value))) {
                unsigned passes = 0;
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (!(v[j][i] < top.bar_value))
                            passes |= 1u << (j * V + i);
                // one candidate of each lane at a time, read again: few pass
                while (__any_sync(0xffffffffu, passes != 0)) {
                    Key k = 0;
                    if (passes) {
                        const int bit = __ffs(passes) - 1;
                        passes &= passes - 1;
                        const int q = q0 + bit / V * kThreads + lane;
                        const int e = q * V - shift + bit % V;
                        if (q < last && e >= 0 && e < p.vocab)
                            k = make_key(Elem<T>::get(x[e]), e);
                    }
                    top.add(k > top.bar, k, p.top);
                }
            }
        }
    }
    if (TOP)
        top.finish();
    a = lanes_join<32>(a);
    if (WARPS > 1) {
        if (lane == 0)
            stats[warp] = a;
        if (TOP)
            lists[warp][lane] = top.list;
        __syncthreads();
        if (warp == 0) {
            a = lanes_join<32>(lane < WARPS ? stats[lane] : Stats{-kInf, 0.0f, 0.0f});
            if (TOP)
                for (int k = 1; k < WARPS; ++k)
                    top.list = warp_merge(top.list, lists[k][31 - lane]);
        }
    }
    if (blocks > 1) {
        ptx::cluster_wait_acquire();  // every block of the cluster runs
        if (warp == 0) {
            if (TOP && rank != 0)
                store_cluster(ptx::map_to_rank(ptx::smem_u32(&block_lists[rank][lane]), 0), top.list);
            if (lane == 0 && rank != 0) {
                const uint32_t at = ptx::map_to_rank(ptx::smem_u32(block_stats[rank]), 0);
                store_cluster(at, static_cast<unsigned long long>(__float_as_uint(a.s)) << 32 |
                                      __float_as_uint(a.m));
                store_cluster(at + 8, __float_as_uint(a.w));
            }
        }
        ptx::cluster_arrive_release();
        ptx::cluster_wait_acquire();
        if (rank != 0)
            return;
        if (warp == 0) {
            Stats b = a;
            if (lane > 0)
                b = lane < blocks ? Stats{block_stats[lane][0], block_stats[lane][1],
                                          block_stats[lane][2]}
                                  : Stats{-kInf, 0.0f, 0.0f};
            a = lanes_join<32>(b);
            if (TOP)
                for (int k = 1; k < blocks; ++k)
                    top.list = warp_merge(top.list, block_lists[k][31 - lane]);
        }
    }
    if (warp != 0)
        return;
    const float ln_s = logf(a.s);
    if (lane == 0)
        write_stats(p, row, a, ln_s, given);
    if (TOP && lane < p.top)
        write_top(p, row, lane, top.list, a, ln_s);
}

template <typename T, int LANES>
int launch_small(const LogprobArgs &p, cudaStream_t stream)
{
    const int st = check_launch_injection("lstm_token_logprobs");
    if (st != LSTM_OK)
        return st;
    const int per_block = kSmallThreads / LANES;
    small_kernel<T, LANES><<<(p.rows + per_block - 1) / per_block, kSmallThreads, 0, stream>>>(p);
    return cuda_status(cudaGetLastError(), "lstm_token_logprobs launch");
}

template <typename T, int WARPS>
int launch_rows(const LogprobArgs &p, int cluster, cudaStream_t stream)
{
    const int st = check_launch_injection("lstm_token_logprobs");
    if (st != LSTM_OK)
        return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.rows, cluster);
    cfg.blockDim = dim3(WARPS * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = cluster;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_status(p.top ? cudaLaunchKernelEx(&cfg, row_kernel<T, WARPS, true>, p)
                             : cudaLaunchKernelEx(&cfg, row_kernel<T, WARPS, false>, p),
                       "lstm_token_logprobs launch");
}

template <typename T>
int launch_typed(const LogprobArgs &p, cudaStream_t stream)
{
    if (p.vocab <= 8)
        return launch_small<T, 8>(p, stream);
    if (p.vocab <= 32)
        return launch_small<T, 32>(p, stream);
    if (p.vocab <= 2048)
        return launch_rows<T, 1>(p, 1, stream);
    // as many blocks a row as it takes to occupy the 152 SMs four blocks deep,
    // each with at least two batches of work
    int cluster = 1;
    while (cluster < kMaxCluster && static_cast<long long>(p.rows) * cluster < 152 * 4 &&
           p.vocab / (cluster * 2) >= 2 * kBatch * Elem<T>::kVector * 256)
        cluster *= 2;
    return launch_rows<T, 8>(p, cluster, stream);
}

}  // namespace
}  // namespace lstm

using namespace lstm;

extern "C" int lstm_token_logprobs(const void *logits, long long stride, int dtype, int rows,
                                   int vocab, const long long *tokens, float *logp, float *entropy,
                                   int top, float *top_logp, long long *top_ids, void *stream)
{
    const char *what = "lstm_token_logprobs";
    int st;
    if ((st = check_dtype(what, dtype)))
        return st;
    if (rows < 0 || vocab <= 0)
        return fail(LSTM_E_INVALID, "%s: %d rows, %d logits a row", what, rows, vocab);
    if (vocab > 1 << 30)
        return fail(LSTM_E_OVERFLOW, "%s: %d logits a row", what, vocab);
    if (top < 0 || top > LSTM_TOP_MAX || top > vocab)
        return fail(LSTM_E_INVALID, "%s: %d alternatives of %d (at most %d)", what, top, vocab,
                    LSTM_TOP_MAX);
    if (!tokens != !logp)
        return fail(LSTM_E_INVALID, "%s: tokens and logp go together", what);
    if (rows == 0)
        return LSTM_OK;
    if ((st = check_matrix(what, "logits", logits, stride, rows, vocab, element_size(dtype))) ||
        (top && ((st = check_matrix(what, "top_logp", top_logp, top, rows, top, 4)) ||
                 (st = check_matrix(what, "top_ids", top_ids, top, rows, top, 8)))))
        return st;
    int device = 0;
    if ((st = op_device(logits, &device)))
        return st;
    DeviceGuard guard(device);
    if (!guard.ok)
        return fail(LSTM_E_CUDA, "cannot make device %d current", device);
    LogprobArgs p = {logits, stride, tokens, logp, entropy, top, top_logp, top_ids, rows, vocab};
    LSTM_WITH_TYPE(dtype, T, return launch_typed<T>(p, static_cast<cudaStream_t>(stream)));
}
