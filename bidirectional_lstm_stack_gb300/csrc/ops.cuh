// Helpers shared by the state-space layer's and the log probabilities'
// kernels (conv.cu, scan.cu, norm.cu, logprobs.cu): element types and their
// vectors, the sequences of a packed batch, the states' slots, and the
// argument checks that the entry points of lstm_ops.h have in common.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "common.cuh"
#include "lstm_ops.h"

namespace lstm {

// ---- host: argument checks ---------------------------------------------------
inline int element_size(int dtype) { return dtype == LSTM_F32 ? 4 : 2; }

inline int check_dtype(const char *what, int dtype)
{
    if (dtype != LSTM_F32 && dtype != LSTM_BF16 && dtype != LSTM_F16)
        return fail(LSTM_E_INVALID, "%s: unknown element type %d", what, dtype);
    return LSTM_OK;
}

// A device matrix argument: element-aligned, rows of `cols` elements.
inline int check_matrix(const char *what, const char *name, const void *p, long long stride,
                        long long rows, long long cols, int size)
{
    if (!p)
        return fail(LSTM_E_INVALID, "%s: %s is null", what, name);
    if (reinterpret_cast<uintptr_t>(p) % size)
        return fail(LSTM_E_INVALID, "%s: %s (%p) is not aligned to its elements", what, name, p);
    if (rows > 1 && stride < cols)
        return fail(LSTM_E_INVALID, "%s: %s has row stride %lld, rows of %lld", what, name, stride,
                    cols);
    return LSTM_OK;
}

// Whether every row of the matrix starts on a multiple of `bytes` (a power of two).
inline bool rows_aligned(const void *p, long long stride, int size, int bytes = 16)
{
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0 && stride * size % bytes == 0;
}

// The most tokens and sequences of a call.  Kernels count both in 32 bits: token
// numbers a tile beyond the last, the sum of two sequence numbers (tile_owner's
// bisection) and a sequence number some grids beyond the last must stay below 2^31.
constexpr int kMostTokens = 0x7fffff00;
constexpr int kMostSequences = LSTM_MAX_SEQUENCES;

inline int check_sequences(const char *what, int tokens, int sequences, const int *offsets)
{
    if (tokens < 0 || sequences < 0 || (tokens > 0 && sequences == 0))
        return fail(LSTM_E_INVALID, "%s: %d tokens, %d sequences", what, tokens, sequences);
    if (tokens > kMostTokens || sequences > kMostSequences)
        return fail(LSTM_E_OVERFLOW, "%s: %d tokens, %d sequences (at most %d, %d)", what, tokens,
                    sequences, kMostTokens, kMostSequences);
    if (!offsets && sequences > 0 && tokens % sequences)
        return fail(LSTM_E_LENGTH,
                    "%s: %d tokens are no multiple of %d sequences (and no offsets are given)", what,
                    tokens, sequences);
    return LSTM_OK;
}

// The device of pointer p made ready for the library's kernels.  Remembers
// per host thread which devices are ready, so that a call costs no lock.
inline int op_device(const void *p, int *device)
{
    int st = pointer_device(p, device);
    if (st != LSTM_OK)
        return st;
    thread_local unsigned long long ready = 0;
    if (*device >= 0 && *device < 64 && (ready >> *device & 1))
        return LSTM_OK;
    if ((st = prepare_device(*device)) == LSTM_OK)
        ready |= 1ull << *device;
    return st;
}

// Remembers on which devices a kernel may use more dynamic shared memory than
// 48 KiB.
struct SharedMemory {
    std::atomic<unsigned long long> done{0};
    template <typename K>
    int allow(K kernel, size_t bytes)
    {
        if (bytes <= 48 * 1024)
            return LSTM_OK;
        int device = 0;
        int st = cuda_status(cudaGetDevice(&device), "current device");
        if (st != LSTM_OK || (done.load() >> device & 1))
            return st;
        st = cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              static_cast<int>(bytes)),
                         "shared memory attribute");
        if (st == LSTM_OK)
            done.fetch_or(1ull << device);
        return st;
    }
};

// A launch as the programmatic dependent of the kernel before it on the stream: its blocks
// may start when that kernel's have all asked for it or ended, and call
// ptx::griddep_wait() before they touch what that kernel reads or writes.
struct Dependent {
    cudaLaunchConfig_t config = {};
    cudaLaunchAttribute attributes[2];
    Dependent(dim3 grid, dim3 block, size_t shared, cudaStream_t stream)
    {
        config.gridDim = grid;
        config.blockDim = block;
        config.dynamicSmemBytes = shared;
        config.stream = stream;
        attributes[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attributes[0].val.programmaticStreamSerializationAllowed = 1;
        config.attrs = attributes;
        config.numAttrs = 1;
    }
    Dependent(const Dependent &) = delete;
};

// ---- sequences and states ------------------------------------------------------
// The sequences of a packed batch, as lstm_ops.h describes them.
struct Sequences {
    const int *offsets;  // null: all of `length` rows
    int count;
    int length;
    int tokens;
};

// Where each sequence keeps its state.
struct Slots {
    const int *slots;   // null: slot s
    const int *resume;  // null: none goes on
    int count;          // 0: no states
};

typedef unsigned long long Pair;  // two fp32 numbers in one 64-bit register

#ifdef __CUDACC__

__device__ __forceinline__ int sequence_begin(const Sequences &q, int s)
{
    if (!q.offsets)
        return s * q.length;
    return min(max(__ldg(q.offsets + s), 0), q.tokens);
}
__device__ __forceinline__ int sequence_end(const Sequences &q, int s)
{
    if (!q.offsets)
        return (s + 1) * q.length;
    return min(max(__ldg(q.offsets + s + 1), sequence_begin(q, s)), q.tokens);
}

// The slot of sequence s, or -1.
__device__ __forceinline__ int sequence_slot(const Slots &p, int s)
{
    if (p.count == 0)
        return -1;
    const int slot = p.slots ? __ldg(p.slots + s) : s;
    return slot >= 0 && slot < p.count ? slot : -1;
}
__device__ __forceinline__ bool sequence_resumes(const Slots &p, int s)
{
    return p.resume && __ldg(p.resume + s) != 0;
}

// Sequence-aligned tiles of `tile` rows.  Sequence s owns the tile numbers
// from base(s) = begin(s) / tile + s on: base(s + 1) - base(s) is at least
// the tiles its rows need and at least one, so the tile numbers below
// tiles_bound() cover every sequence, and the owner of a tile is found by
// bisection over the offsets alone (a few numbers own no rows).  Lengths need
// not be known on the host.
__host__ __device__ inline long long tiles_bound(int tokens, int sequences, int tile)
{
    return tokens / tile + static_cast<long long>(sequences);
}
__device__ __forceinline__ int tile_owner(const Sequences &q, int number, int tile, int *first)
{
    int lo = 0, hi = q.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sequence_begin(q, mid) / tile + mid <= number)
            lo = mid;
        else
            hi = mid - 1;
    }
    *first = number - (sequence_begin(q, lo) / tile + lo);
    return lo;
}

// ---- element types ---------------------------------------------------------------
template <typename T>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int kVector = 4;  // elements in 16 bytes
    static __device__ __forceinline__ float get(float v) { return v; }
    static __device__ __forceinline__ float put(float v) { return v; }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int kVector = 8;
    static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<__half> {
    static constexpr int kVector = 8;
    static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};

// V consecutive elements: 1, or the 16 bytes of an aligned vector.
template <typename T, int V>
struct alignas(V * sizeof(T)) Pack {
    T v[V];
};
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T *p)
{
    Pack<T, V> r;
    if constexpr (V * sizeof(T) == 16)
        *reinterpret_cast<uint4 *>(&r) = __ldg(reinterpret_cast<const uint4 *>(p));
    else
        r = *reinterpret_cast<const Pack<T, V> *>(p);
    return r;
}
template <typename T, int V>
__device__ __forceinline__ void store_pack(T *p, const Pack<T, V> &r)
{
    *reinterpret_cast<Pack<T, V> *>(p) = r;
}
template <typename T, int V>
__device__ __forceinline__ void unpack(const Pack<T, V> &r, float (&f)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i)
        f[i] = Elem<T>::get(r.v[i]);
}
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> pack(const float (&f)[V])
{
    Pack<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i)
        r.v[i] = Elem<T>::put(f[i]);
    return r;
}

// V consecutive fp32 weights, 16-byte aligned where V is a multiple of 4.
template <int V>
__device__ __forceinline__ void load_weights(const float *p, float (&w)[V])
{
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<float4 *>(w + i) = __ldg(reinterpret_cast<const float4 *>(p + i));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            w[i] = __ldg(p + i);
    }
}

// ---- functions ---------------------------------------------------------------------
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// 1 / x for x not below fp32's normal range (infinity gives 0).
__device__ __forceinline__ float reciprocal(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// v / (1 + e^-v): e^-v saturates to 0 or infinity, and the quotient by an
// infinity is 0.
__device__ __forceinline__ float silu(float v)
{
    return v * reciprocal(1.0f + ex2(-kLog2e * v));
}

// ---- pairs -------------------------------------------------------------------------
// The paired operations do two roundings each in one issue slot.  They are
// volatile so that the compiler keeps them in the order they are written in,
// which hides their latencies.
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
    asm volatile("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b)
{
    Pair r;
    asm volatile("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c)
{
    Pair r;
    asm volatile("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ Pair ex2_pair(Pair p)
{
    const float2 v = split_pair(p);
    float x, y;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(v.x));
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v.y));
    return make_pair(x, y);
}
__device__ __forceinline__ Pair reciprocal_pair(Pair p)
{
    const float2 v = split_pair(p);
    float x, y;
    asm volatile("rcp.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(v.x));
    asm volatile("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v.y));
    return make_pair(x, y);
}

// v / (1 + e^-v) in place for K pairs, side by side, so that none waits for its
// own result
template <int K>
__device__ __forceinline__ void silu_pairs(Pair (&v)[K])
{
    Pair e[K];
#pragma unroll
    for (int k = 0; k < K; ++k)
        e[k] = mul2(v[k], make_pair(-kLog2e, -kLog2e));
#pragma unroll
    for (int k = 0; k < K; ++k)
        e[k] = add2(ex2_pair(e[k]), make_pair(1.0f, 1.0f));
#pragma unroll
    for (int k = 0; k < K; ++k)
        v[k] = mul2(v[k], reciprocal_pair(e[k]));
}

// ---- parts of bf16 -----------------------------------------------------------------
// Two numbers rounded to bf16, in one register.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Those beyond bf16's largest number, infinities too, give it.
__device__ __forceinline__ uint32_t bf16_pair_finite(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float low_float(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float high_float(uint32_t pair)
{
    return __uint_as_float(pair & 0xffff0000u);
}
// Two numbers as N pairs of parts, each the rest's nearest.  Three are the whole fp32 number (down
// to 2^-133, where bf16 ends), and the rests have either sign: of two numbers' nine products of
// parts the three smallest are 2^-24 of the whole at most and point all ways.  (Parts cut off
// instead of rounded lose 2^-21, always towards zero.)  An infinity's are bf16's largest number,
// an infinity and (of three) a NaN.
template <int N>
__device__ __forceinline__ void split_pair_parts(float x, float y, uint32_t (&r)[N])
{
#pragma unroll
    for (int k = 0; k < N; ++k) {
        // (fp32 numbers next to the largest would round to infinity)
        r[k] = N > 1 && k == 0 ? bf16_pair_finite(x, y) : bf16_pair(x, y);
        if (k + 1 < N) {
            x -= low_float(r[k]);
            y -= high_float(r[k]);
        }
    }
}

template <typename F>
__device__ __forceinline__ float warp_reduce(float v, F f)
{
#pragma unroll
    for (int m = 16; m; m >>= 1)
        v = f(v, __shfl_xor_sync(0xffffffffu, v, m));
    return v;
}

#endif  // __CUDACC__

// Runs the statement with T as dtype's element type.
#define LSTM_WITH_TYPE(dtype, T, ...)        \
    do {                                     \
        if ((dtype) == LSTM_F32) {           \
            using T = float;                 \
            __VA_ARGS__;                     \
        } else if ((dtype) == LSTM_BF16) {   \
            using T = __nv_bfloat16;         \
            __VA_ARGS__;                     \
        } else {                             \
            using T = __half;                \
            __VA_ARGS__;                     \
        }                                    \
    } while (0)

}  // namespace lstm
