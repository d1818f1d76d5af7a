// Log probabilities of given tokens, the entropy and the top alternatives of
// rows of logits, in one pass over the logits.
//
// A row's softmax is summed while it streams by: with m the largest logit so
// far, s = sum e^(x - m) and w = sum e^(x - m) (x - m) are scaled by e^(m - m')
// whenever m grows to m', and at the end
//   l[v] = (x[v] - m) - ln s,   entropy = ln s - w / s.
// The top alternatives are 64-bit keys, the logit's order above the index's, so
// that equal logits rank by index and no order of work changes the result.
// While the row streams by, only each thread's largest logits are kept; they
// give a bar that enough logits reach, the few vectors with logits above it are
// looked at again (from the caches), and the keys found are put in order by
// counting, for each, the keys above it.  Long rows are shared by the blocks of
// a cluster, which join their sums and keys through distributed shared memory.
//
// 64 rows of 100003 bf16: 6.4 us without alternatives, 13 us with 20 (their bytes
// take 1.9 us at the card's copy rate); 2048 rows of 32000: 35 us (3.8 TB/s) and
// 51 us (19 us).  Neither the bytes nor the instructions bound it: some eight an
// element would take 14 us for the latter rows.  It waits: a turn's loads are
// issued only after the last turn's sums, and nothing is loaded between the
// barriers of the joins and of the selection (with 20 alternatives issue slots are
// 48 % busy, barriers and loads the longest stalls).
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
// The Stats of all lanes together.
__device__ __forceinline__ Stats lanes_join(Stats a)
{
    float m = a.m;
#pragma unroll
    for (int i = 16; i; i >>= 1)
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, i));
    a = rescale(a, m);
#pragma unroll
    for (int i = 16; i; i >>= 1) {
        a.s += __shfl_xor_sync(0xffffffffu, a.s, i);
        a.w += __shfl_xor_sync(0xffffffffu, a.w, i);
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
// (Not inlined, like absorb: a call's warps run this code only a few times, so
// its size counts, which they wait for to be fetched.)
__device__ __noinline__ Key warp_merge(Key list, Key ascending)
{
    Key k = list > ascending ? list : ascending;  // bitonic
#pragma unroll
    for (int step = 16; step; step >>= 1)
        k = exchange(k, step, (threadIdx.x & step) == 0);
    return k;
}
// The same for 32 other keys in any order.
__device__ __noinline__ Key warp_absorb(Key list, Key any)
{
    return warp_merge(list, lanes_sort<32, true>(any));
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
    if (LANES == 32) {
        // the largest left, again and again; the lowest lane of equals
        unsigned u = i < p.vocab ? static_cast<unsigned>(make_key(v, 0) >> 32) : 0;
        for (int j = 0; j < p.top; ++j) {
            const unsigned most = __reduce_max_sync(0xffffffffu, u);
            const unsigned who = __ballot_sync(0xffffffffu, u == most);
            if (i == __ffs(who) - 1) {
                if (live)
                    write_top(p, row, j, make_key(v, i), a, ln_s);
                u = 0;
            }
        }
    } else if (p.top) {
        // a lane's rank: how many keys are above its own
        const Key k = i < p.vocab ? make_key(v, i) : 0;
        int above = 0;
#pragma unroll
        for (int j = 1; j < LANES; ++j)
            above += __shfl_xor_sync(0xffffffffu, k, j) > k;
        if (live && i < p.vocab && above < p.top)
            write_top(p, row, above, k, a, ln_s);
    }
}

// ---- longer rows: WARPS warps of each of a cluster's blocks a row ----------------
// A thread's batch: 32 elements in 16-byte vectors, loaded together.
constexpr int kBatchElements = 32;
constexpr int kMaxCluster = 8;
constexpr int kListed = 1024;

// A warp's running top list and its candidates.
struct TopList {
    Key list;         // lane i: the i-th largest so far
    Key bar;          // only keys above it matter
    float bar_value;  // its logit; -infinity without a bar
    int waiting;      // candidates in the buffer, fewer than 32 between calls
    Key *buffer;      // 63 keys of shared memory

    __device__ __forceinline__ void raise(Key k)
    {
        if (k > bar) {
            bar = k;
            bar_value = key_value(k);
        }
    }
    // Takes the lanes' keys that are above the bar.
    __device__ __forceinline__ void add(Key k, int top)
    {
        const unsigned mask = __ballot_sync(0xffffffffu, k > bar);
        const int lane = threadIdx.x % 32;
        if (k > bar)
            buffer[waiting + __popc(mask & ((1u << lane) - 1))] = k;
        waiting += __popc(mask);
        __syncwarp();
        if (waiting >= 32)
            merge(top);
    }
    // Merges up to 32 of the waiting keys.
    __device__ __forceinline__ void merge(int top)
    {
        const int lane = threadIdx.x % 32, take = min(waiting, 32);
        const Key k = lane < take ? buffer[waiting - take + lane] : 0;
        __syncwarp();
        waiting -= take;
        list = warp_absorb(list, k);
        raise(__shfl_sync(0xffffffffu, list, top - 1));
    }
};

// The largest of the block's `total` different keys in `all` (16-byte aligned,
// with room for kPad keys behind them), in order: result[i] is the i-th largest,
// 0 beyond them.  A key's place is the number of keys above it, which its thread
// counts.  All threads call it, after a barrier behind the keys; ends with one.
constexpr int kPad = 16;
template <int THREADS>
__device__ __forceinline__ void order_keys(Key *all, int total, Key (&result)[32])
{
    if (threadIdx.x < 32)
        result[threadIdx.x] = 0;
    if (threadIdx.x < kPad)
        all[total + threadIdx.x] = 0;
    __syncthreads();
    for (int at = threadIdx.x; at < total; at += THREADS) {
        const Key k = all[at];
        int above = 0;
        for (int j = 0; j < total; j += kPad) {
            ulonglong2 two[kPad / 2];
#pragma unroll
            for (int i = 0; i < kPad / 2; ++i)
                two[i] = *reinterpret_cast<const ulonglong2 *>(all + j + 2 * i);
#pragma unroll
            for (int i = 0; i < kPad / 2; ++i)
                above += (two[i].x > k) + (two[i].y > k);
        }
        if (k && above < 32)
            result[above] = k;
    }
    __syncthreads();
}

__device__ __forceinline__ void store_cluster(uint32_t addr, unsigned long long v)
{
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

template <typename T, int WARPS, bool TOP>
__global__ void __launch_bounds__(WARPS * 32, WARPS == 8 ? 4 : 24 / WARPS) row_kernel(LogprobArgs p)
{
    constexpr int V = Elem<T>::kVector, kBatch = kBatchElements / V;
    constexpr int kThreads = WARPS * 32;
    __shared__ Key buffers[TOP ? WARPS : 1][64];
    // all warps' keys: their lists and what waits in their buffers
    __shared__ __align__(16) Key all[TOP ? WARPS * 64 + kPad : 1];
    __shared__ Key result[32];
    __shared__ unsigned bars[WARPS];
    __shared__ int listed;
    __shared__ int list[TOP ? kListed : 1];
    __shared__ int counts[WARPS];
    __shared__ Stats stats[WARPS];
    // what the cluster's blocks send to its first
    __shared__ __align__(16) Key block_keys[TOP ? kMaxCluster * 32 + kPad : 1];
    __shared__ __align__(16) float block_stats[kMaxCluster][4];
    const uint32_t rank = ptx::cluster_ctarank();
    const int blocks = gridDim.y;  // the cluster's
    const int row = blockIdx.x;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    if (blocks > 1)
        ptx::cluster_arrive_release();
    if (threadIdx.x == 0)
        listed = 0;
    const T *x = static_cast<const T *>(p.logits) + row * p.stride;
    const float given = threadIdx.x == 0 && rank == 0 ? token_logit(p, x, row) : 0.0f;
    // the row in 16-byte vectors of its own alignment: vector q holds the
    // elements q * V - shift .. + V-1, the first and the last partly outside
    const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    const int vectors = static_cast<int>((static_cast<long long>(p.vocab) + shift + V - 1) / V);
    const int share = (vectors + blocks - 1) / blocks;
    const int first = min(vectors, static_cast<int>(rank) * share);
    const int last = min(vectors, first + share);

    float column[kBatch];  // the largest logit of the batches' j-th vectors
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
        column[j] = -kInf;
    float a_m = -kInf;
    Pair s2 = 0, w2 = 0;  // s and w of Stats, of the even and of the odd elements
    TopList top = {0, 0, -kInf, 0, buffers[TOP ? warp : 0]};
    // (all warps take the same turns)
    const auto read = [&](int q, float (&v)[V]) {  // absent elements: -infinity
        const int e0 = q * V - shift;
        if (q < last && e0 >= 0 && e0 + V <= p.vocab) {
            unpack<T, V>(load_pack<T, V>(x + e0), v);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[i] = -kInf;
            if (q < last) {  // the row's ends
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (e0 + i >= 0 && e0 + i < p.vocab)
                        v[i] = Elem<T>::get(x[e0 + i]);
            }
        }
    };
    for (int q0 = first; q0 < last; q0 += kBatch * kThreads) {
        float v[kBatch][V];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            read(q0 + j * kThreads + static_cast<int>(threadIdx.x), v[j]);
        float m = a_m;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            float most = v[j][0];
#pragma unroll
            for (int i = 1; i < V; ++i)
                most = max_nan(most, v[j][i]);
            if (TOP)
                column[j] = max_nan(column[j], most);
            m = max_nan(m, most);
        }
        if (!(m == a_m)) {
            const float f = ex2((a_m - m) * kLog2e);
            // nothing summed, or nothing left of it: also where a_m - m is infinite
            if (a_m == -kInf || f == 0.0f) {
                s2 = w2 = 0;
            } else {
                w2 = mul2(fma2(s2, make_pair(a_m - m, a_m - m), w2), make_pair(f, f));
                s2 = mul2(s2, make_pair(f, f));
            }
            a_m = m;
        }
        const float base = m == -kInf ? 0.0f : -m;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            // (a whole warp beyond the end has nothing to add)
            if (q0 + j * kThreads + warp * 32 >= last)
                break;
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                const Pair d = add2(make_pair(v[j][i], v[j][i + 1]), make_pair(base, base));
                const Pair e = ex2_pair(mul2(d, make_pair(kLog2e, kLog2e)));
                const float2 d2 = split_pair(d);
                s2 = add2(s2, e);
                // (a difference of -infinity would make a NaN of 0)
                w2 = fma2(e, make_pair(fmaxf(d2.x, -1e30f), fmaxf(d2.y, -1e30f)), w2);
            }
        }
    }
    if (TOP) {
        // A bar that `top` of the block's logits reach: the smallest of the
        // warps' n-th largest lane maxima, with n lanes of every warp enough.
        const int each = (p.top + WARPS - 1) / WARPS;
        const bool some = first + static_cast<int>(threadIdx.x) < last;
        unsigned u = some ? static_cast<unsigned>(make_key(a_m, 0) >> 32) : 0, nth = 0;
        for (int k = 0; k < each; ++k) {
            nth = __reduce_max_sync(0xffffffffu, u);
            const unsigned who = __ballot_sync(0xffffffffu, u == nth);
            if (lane == __ffs(who) - 1)
                u = 0;
        }
        if (lane == 0)
            bars[warp] = nth;
        __syncthreads();
        if (WARPS > 1) {
#pragma unroll
            for (int k = 0; k < WARPS; ++k)
                nth = min(nth, bars[k]);
        }
        // below every key of that logit; none where a warp lacks lanes
        if (nth)
            top.raise(static_cast<Key>(nth) << 32);
        // Few of the threads' columns of vectors (the j-th ones of its batches)
        // have logits above it: they are listed, and the warps share out a
        // second look at the listed vectors, an element a lane.  (In any order:
        // none changes the result.)
        const int batches = (last - first + kBatch * kThreads - 1) / (kBatch * kThreads);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int q0 = first + j * kThreads + static_cast<int>(threadIdx.x);
            const bool flag = q0 < last && !(column[j] < top.bar_value);
            const unsigned mask = __ballot_sync(0xffffffffu, flag);
            if (!mask)
                continue;
            int at = 0;
            if (lane == 0)
                at = atomicAdd(&listed, __popc(mask) * batches);
            at = __shfl_sync(0xffffffffu, at, 0) + __popc(mask & ((1u << lane) - 1)) * batches;
            if (flag && at + batches <= kListed)
                for (int k = 0; k < batches; ++k)
                    list[at + k] = q0 + k * kBatch * kThreads;
        }
        __syncthreads();
        // too many for the list (rows of equal logits): a look at all
        const bool some_only = listed <= kListed;
        const int items = some_only ? listed : last - first;
        constexpr int kVectors = 32 / V, kLooks = 4;  // vectors of a look, looks at a time
        for (int i0 = warp * kVectors; i0 < items; i0 += WARPS * kVectors * kLooks) {
            float v[kLooks];
            int e[kLooks];
#pragma unroll
            for (int k = 0; k < kLooks; ++k) {
                const int i = i0 + k * WARPS * kVectors + lane / V;
                const int q = i >= items ? last : some_only ? list[i] : first + i;
                e[k] = q * V - shift + lane % V;
                const bool in = q < last && e[k] >= 0 && e[k] < p.vocab;
                v[k] = in ? Elem<T>::get(x[e[k]]) : -kInf;
                e[k] = in ? e[k] : -1;
            }
#pragma unroll
            for (int k = 0; k < kLooks; ++k)
                if (__any_sync(0xffffffffu, !(v[k] < top.bar_value)))
                    top.add(e[k] >= 0 ? make_key(v[k], e[k]) : 0, p.top);
        }
    }
    const float2 s_parts = split_pair(s2), w_parts = split_pair(w2);
    Stats a = lanes_join({a_m, s_parts.x + s_parts.y, w_parts.x + w_parts.y});
    if (WARPS > 1) {
        // a warp has a list only if it has merged anything
        const int keys = top.waiting + (top.list != 0 ? 32 : 0);
        if (lane == 0) {
            stats[warp] = a;
            counts[warp] = keys;
        }
        __syncthreads();
        if (warp == 0)
            a = lanes_join(lane < WARPS ? stats[lane] : Stats{-kInf, 0.0f, 0.0f});
        if (TOP) {
            int total = 0, before = 0;
#pragma unroll
            for (int k = 0; k < WARPS; ++k) {
                before += k < warp ? counts[k] : 0;
                total += counts[k];
            }
            if (lane < top.waiting)
                all[before + lane] = top.buffer[lane];
            if (keys >= 32)
                all[before + top.waiting + lane] = top.list;
            order_keys<kThreads>(all, total, result);
            top.list = result[lane];
        }
    } else if (TOP && top.waiting) {
        top.merge(p.top);
    }
    if (blocks > 1) {
        ptx::cluster_wait_acquire();  // every block of the cluster runs
        if (warp == 0) {
            if (TOP && lane < p.top)
                store_cluster(
                    ptx::map_to_rank(ptx::smem_u32(&block_keys[rank * p.top + lane]), 0), top.list);
            if (lane == 0) {
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
        if (warp == 0)
            a = lanes_join(lane < blocks ? Stats{block_stats[lane][0], block_stats[lane][1],
                                                     block_stats[lane][2]}
                                             : Stats{-kInf, 0.0f, 0.0f});
        if (TOP) {
            order_keys<kThreads>(block_keys, blocks * p.top, result);
            top.list = result[lane];
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
    const unsigned blocks = (static_cast<unsigned>(p.rows) + per_block - 1) / per_block;
    small_kernel<T, LANES><<<blocks, kSmallThreads, 0, stream>>>(p);
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
    // (4096 rows of 1000 bf16, 20 alternatives: 1 warp a row 25 us, 2 warps 19,
    // 4 warps 21; of 200: 21, 27 and 44)
    if (p.vocab <= 512)
        return launch_rows<T, 1>(p, 1, stream);
    if (p.vocab <= 4096)
        return launch_rows<T, 2>(p, 1, stream);
    // as many blocks a row as the SMs hold at once (four each), each thread
    // with a batch at least
    int cluster = 1;
    while (cluster < kMaxCluster && static_cast<long long>(p.rows) * cluster * 2 <= 152 * 4 &&
           p.vocab / cluster >= kBatchElements * 256)
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
