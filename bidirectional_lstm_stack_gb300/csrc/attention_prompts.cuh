// Linear attention over prompts, in chunks of 64 tokens on the tensor cores.  With c_i
// the sum of the chunk's log decays up to token i and S the state before it,
//     y_i = scale (e^(c_i) S^T q_i + sum_(j <= i) e^(c_i - c_j) (q_i . k_j) v_j)
//     S'  = e^(c_64) S + sum_j e^(c_64 - c_j) k_j v_j^T.
// A CTA takes one head of one run of tokens and up to 128 of its values, and keeps S
// transposed: tensor-memory lanes are values, so every product has M = 128 lanes and no
// state ever goes through shared memory.  Per chunk the tensor cores make
//     scores   Q K^T            [64 queries x 64 keys]   (lanes are queries)
//     inter    S^T Q^T          [values x 64 queries]    (S^T in tensor memory)
//     intra    V^T P^T          [values x 64 queries]    (P: decayed, masked scores)
//     update   (wV)^T K         [values x keys]          (w_j = e^(c_64 - c_j))
// and the warps have one task each:
//  * bf16 rows that start on 16-byte boundaries come by TMA (128-byte swizzle, so the same
//    tile serves as K-major and as MN-major operand), asked for by one thread; others are
//    read, split into parts and written by 4 loaders.  A ring of up to three stages;
//  * a warp sums the log decays, as pairs of fp32 numbers: c_i - c_j of far sums would lose
//    what separates near tokens;
//  * 3 warps turn scores into P, 4 others inter and intra into y, a chunk behind;
//  * 4 or 8 state warps hold S in registers (fp32, a lane per value), add the update and hand
//    S on as parts of bf16;
//  * with TMA the loaders' warps write w v of the next chunk, else the state warps do;
//  * two threads issue the products, those of the outputs and those of the states, so that
//    neither chain waits for the other.
// Where sequences and heads are fewer than SMs, sequences are cut into spans: a first pass
// makes what each span adds to a state of zeros (no outputs), a small kernel joins them to
// the states that the spans start from, and then all spans run side by side.
// bf16 inputs are exact operands.  P and S go as two parts of bf16 for their products, 2^-17 of
// them off, where an output of 16 bits is rounded to 2^-8 or 2^-11 itself (with one part y was off
// by 2.35e-3 of its norm, 1.66e-3 of which are its own rounding, and a prompt's outputs were not
// its single tokens'; a chunk took 1.97 us then and takes 2.42).  w v goes as three parts, so that
// what joins the state, which is fp32, keeps 24 bits (two parts left 2.4e-6 of it).  fp16 inputs
// are two parts of bf16 (exact; P and S in fp16 itself would overflow); fp32 three parts (exact),
// and so are P and S.  Of two factors' parts those products are made that the other roundings
// leave visible (parts a, b with a + b below the larger number of parts).
//
// What bounds it: with bf16 and 128 keys and values a chunk's products keep the tensor core busy
// for 1 790 cycles, its instructions the ALU pipe for 1 780; the warps' chains, whose instructions
// exceed the instruction cache, make it 5 000.  fp16 and fp32 wait for their loaders (13.4 and
// 14.2 us a chunk).  16 heads of a prompt of 4096 tokens take 52 us (68 MB: 10 us), four
// prompts of 16384 tokens 478 us (675 MB: 99 us).  Waits, loops and rare branches are kept
// short for that reason: inlining a wait's clock and messages at its 20 places cost a quarter
// of the time at 64 keys.
#pragma once

#include "attention.cuh"

namespace lstm {
namespace prompts {

constexpr int C = 64;           // tokens of a chunk
constexpr int kRowBytes = 128;  // of a tile's row: 64 bf16
constexpr int kSlab = C * kRowBytes;
constexpr int kMaxStages = 3;
constexpr int kLoaders = 128;
constexpr float kMostDecay = 300.0f;  // log2 of a decay that leaves nothing of any fp32 number

// Parts of bf16 that the numbers of a type are split into.
template <typename T>
struct Parts;
template <>
struct Parts<__nv_bfloat16> {
    static constexpr int kIn = 1, kMid = 2;
};
template <>
struct Parts<__half> {
    static constexpr int kIn = 2, kMid = 2;
};
template <>
struct Parts<float> {
    static constexpr int kIn = 3, kMid = 3;
};
constexpr int kWeighted = 3;  // of w v

// A run of tokens that one CTA takes, and the state it starts from and leaves.
struct Run {
    int begin, end;
    const float *from;  // null: zeros
    float *to;          // null: not kept
};

// Of q, k and v, for TMA.
struct Maps {
    CUtensorMap of[3];
};

// What one stage holds beside its tiles.
struct Decays {
    float2 sum[C];   // c_i in log2, as the fp32 next to it and the rest
    float until[C];  // e^(c_64 - c_i)
};

// What the output and state warps want to know of a chunk, whose stage may be another
// chunk's by then.
// Chunk c + 5 is loaded when y of chunk c is done at the earliest: three stages, and two
// buffers of scores before y.
struct Info {
    float since[C];      // e^(c_i)
    int first_bad[128];  // of a value's column: the first token that is not finite, or C
    float all;           // e^(c_64)
    float pad[3];
};
// Sequences that a block puts in order for itself, which takes it longer the more there are: 24
// prompts with 32 heads of 64 x 64 take 101 us (131 as they come), 128 with 16 heads 156 (160); 160
// would take 190 (173).
constexpr int kOrdered = 128;
constexpr int kInfos = 8;
// Tokens of y that an output warp stores at a time: with 64 there is no room for a third stage at
// 128 keys and values of bf16 (a chunk takes 2.54 us then, 2.42 so), at 64 keys there is (1.65 us,
// 1.87 with 32).
template <int KP>
constexpr int kOutRows = KP == 128 ? 32 : C;
// V's tile is clean: its weighing is two chunks ahead of the outputs at most
constexpr int kCleans = 4;

struct Layout {
    int slabs;         // of v: 64 values each
    int stages;
    int p_buffers;
    int tile_k, tile_v, stage, weighted, p, staging;  // bytes
    size_t total;
};

struct Barriers {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t scores_full[2], p_full[2], inter_full[2], intra_full[2], y_free[2];
    uint64_t weighted_full[2], weighted_free[2];  // of half of the tokens each
    uint64_t clean[kCleans], state_full, update_full, update_free;
    uint64_t done[2];
    uint32_t tmem;
    int abort, sequence;
};

template <typename T, int KP>
Layout layout(int values)
{
    using P = Parts<T>;
    Layout l;
    l.slabs = values > 64 ? 2 : 1;
    l.tile_k = KP / 64 * kSlab;
    l.tile_v = l.slabs * kSlab;
    l.stage = P::kIn * (2 * l.tile_k + l.tile_v);
    l.weighted = kWeighted * l.tile_v;
    l.p = P::kMid * kSlab;
    // y on its way out, 32 values of a row side by side (fp32 rows are as wide as a warp's store)
    l.staging = sizeof(T) == 2 ? 4 * kOutRows<KP> * 32 * 2 : 0;
    // (products of 128 lanes read past tiles of 64, into the tile behind them)
    const size_t rest = l.weighted + l.staging + kMaxStages * sizeof(Decays) + kInfos * sizeof(Info) +
                        sizeof(Barriers) + 1024;
    const auto bytes = [&] { return l.stages * l.stage + l.p_buffers * l.p + rest; };
    // as many stages as there is room for, then a second P
    for (int n = 2 * kMaxStages + 1; n > 1; --n) {
        l.stages = n / 2;
        l.p_buffers = 1 + n % 2;
        if (bytes() <= 227 * 1024)
            break;
    }
    l.total = bytes();
    return l;
}

// ---- parts -----------------------------------------------------------------------------
// Eight numbers as N units of 16 bytes, `apart` bytes from each other.
template <int N>
__device__ __forceinline__ void store_parts(uint8_t *at, int apart, const float (&f)[8])
{
    uint32_t r[4][N];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        split_pair_parts<N>(f[2 * i], f[2 * i + 1], r[i]);
#pragma unroll
    for (int k = 0; k < N; ++k)
        *reinterpret_cast<uint4 *>(at + k * apart) = make_uint4(r[0][k], r[1][k], r[2][k], r[3][k]);
}

// fma2 and mul2 that the compiler may put in any order.
__device__ __forceinline__ Pair free_fma2(Pair a, Pair b, Pair c)
{
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ Pair free_mul2(Pair a, Pair b)
{
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The numbers that N units of 16 bytes stand for, in pairs.
template <int N>
__device__ __forceinline__ void load_parts(const uint8_t *at, int apart, Pair (&f)[4])
{
#pragma unroll
    for (int k = N - 1; k >= 0; --k) {
        const uint4 u = *reinterpret_cast<const uint4 *>(at + k * apart);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Pair some = make_pair(low_float(w[i]), high_float(w[i]));
            f[i] = k == N - 1 ? some : add2(f[i], some);
        }
    }
}

// Four pairs as three units of 16 bytes, their parts.  With ROUND they are split_pair_parts'; cut
// off they have the number's sign, so that a product beyond fp32's range overflows to its side:
// where the other factor is one part, nothing is left out and rounding gains nothing.
template <bool ROUND>
__device__ __forceinline__ void store_three(uint8_t *at, int apart, Pair (&f)[4])
{
    const Pair minus = make_pair(-1.0f, -1.0f);
#pragma unroll
    for (int k = 0; k < kWeighted; ++k) {
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = split_pair(f[i]);
            if (ROUND)
                r[i] = k == 0 ? bf16_pair_finite(v.x, v.y) : bf16_pair(v.x, v.y);
            else
                asm("prmt.b32 %0, %1, %2, 0x7632;"
                    : "=r"(r[i])
                    : "r"(__float_as_uint(v.x)), "r"(__float_as_uint(v.y)));
            if (k + 1 < kWeighted)
                f[i] = free_fma2(make_pair(low_float(r[i]), high_float(r[i])), minus, f[i]);
        }
        *reinterpret_cast<uint4 *>(at + k * apart) = make_uint4(r[0], r[1], r[2], r[3]);
    }
}

// ---- loading ------------------------------------------------------------------------------
// Rows of a head on their way into a tile, 1 << units units of 16 bytes a row (up to 16); rows
// from `len` and numbers from `width` on are zeros, and what lies behind the units stays.  A
// thread keeps its unit and goes down the rows, two at a time, so that swizzle and width are
// worked out once.
constexpr int kTogether = 2;
template <typename T>
__device__ __forceinline__ void read_rows(float (&f)[kTogether][8], const T *from, long long stride,
                                          bool aligned, int len, int width, int units, int group,
                                          int tid)
{
    const int down = kLoaders >> units;  // rows of a turn, a multiple of 8
    const int u = tid & ((1 << units) - 1), r = (tid >> units) + group * kTogether * down;
    const T *src = from + r * stride + u * 8;
    const int there = min(max(width - u * 8, 0), 8);
    if (aligned && there == 8) {
        constexpr int V = Elem<T>::kVector;
#pragma unroll
        for (int k = 0; k < kTogether; ++k)
#pragma unroll
            for (int j = 0; j < 8; j += V) {
                Pack<T, V> v = {};
                if (r + k * down < len)
                    v = load_pack<T, V>(src + k * down * stride + j);
#pragma unroll
                for (int e = 0; e < V; ++e)
                    f[k][j + e] = Elem<T>::get(v.v[e]);
            }
    } else {
#pragma unroll
        for (int k = 0; k < kTogether; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f[k][j] = r + k * down < len && j < there ? Elem<T>::get(src[k * down * stride + j])
                                                          : 0.0f;
    }
}
template <int N>
__device__ __forceinline__ void write_rows(const float (&f)[kTogether][8], uint8_t *tile, int apart,
                                           int units, int group, int tid)
{
    const int down = kLoaders >> units;
    const int u = tid & ((1 << units) - 1), r = (tid >> units) + group * kTogether * down;
    uint8_t *const dst = tile + (u >> 3) * kSlab + r * kRowBytes + (((u & 7) ^ (r & 7)) << 4);
#pragma unroll
    for (int k = 0; k < kTogether; ++k)
        if (r + k * down < C)
            store_parts<N>(dst + k * down * kRowBytes, apart, f[k]);
}

// A sum that fp32 alone would round too early, as the fp32 number next to it and the rest
// (error-free transformation of a sum, Knuth).  This GPU has little fp64.
struct Sum {
    float hi, lo;
};
__device__ __forceinline__ Sum add(Sum a, Sum b)
{
    const float s = a.hi + b.hi, t = s - a.hi;
    const float lo = (a.hi - (s - t)) + (b.hi - t) + (a.lo + b.lo);
    const float hi = s + lo;
    return {hi, lo - (hi - s)};
}
// A log decay in log2 (log2 e = 1.44269502 + 1.92596303e-8), a NaN left as it is.
__device__ __forceinline__ Sum log2_decay(float g)
{
    const float v = g * 1.44269502f;
    if (fabsf(v) > kMostDecay)
        return {v < 0.0f ? -kMostDecay : kMostDecay, 0.0f};
    return {v, fmaf(g, 1.92596303e-8f, fmaf(g, 1.44269502f, -v))};
}

// The sums of a chunk's log decays, two tokens a lane; returns the whole sum.
__device__ __forceinline__ Sum sum_decays(Decays &d, Info &info, float g0, float g1, int lane)
{
    const Sum a = log2_decay(g0), b = log2_decay(g1);
    Sum sum = add(a, b), none = {0.0f, 0.0f};
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
        const Sum other = {__shfl_up_sync(0xffffffffu, sum.hi, m), __shfl_up_sync(0xffffffffu, sum.lo, m)};
        sum = add(sum, lane >= m ? other : none);
    }
    Sum before = {__shfl_up_sync(0xffffffffu, sum.hi, 1), __shfl_up_sync(0xffffffffu, sum.lo, 1)};
    const Sum end = {__shfl_sync(0xffffffffu, sum.hi, 31), __shfl_sync(0xffffffffu, sum.lo, 31)};
    const Sum first = add(lane > 0 ? before : none, a);
    *reinterpret_cast<float4 *>(&d.sum[2 * lane]) = make_float4(first.hi, first.lo, sum.hi, sum.lo);
    *reinterpret_cast<float2 *>(&d.until[2 * lane]) =
        make_float2(ex2((end.hi - first.hi) + (end.lo - first.lo)),
                    ex2((end.hi - sum.hi) + (end.lo - sum.lo)));
    *reinterpret_cast<float2 *>(&info.since[2 * lane]) =
        make_float2(ex2(first.hi) * fmaf(0.6931472f, first.lo, 1.0f),
                    ex2(sum.hi) * fmaf(0.6931472f, sum.lo, 1.0f));
    *reinterpret_cast<int4 *>(&info.first_bad[4 * lane]) = make_int4(C, C, C, C);
    if (lane == 0)
        info.all = ex2(end.hi + end.lo);
    return end;
}

// Values of token j that are not finite, among 8 of its row: zeros take their place in the
// tile, where they would meet the zeros of P at the tokens before j, and their columns'
// first bad token is at most j.
template <int N>
__device__ __forceinline__ void not_finite(uint8_t *at, int apart, int *first_bad, int j)
{
#pragma unroll 1
    for (int e = 0; e < 8; ++e, at += 2) {
        // (an infinity's first part of several is the largest number, the second an infinity)
        const unsigned short tell = *reinterpret_cast<const unsigned short *>(at + (N > 1 ? apart : 0));
        if ((tell & 0x7f80) == 0x7f80) {
            atomicMin(first_bad + e, j);
#pragma unroll
            for (int k = 0; k < N; ++k)
                *reinterpret_cast<unsigned short *>(at + k * apart) = 0;
        }
    }
}

// A number from or to memory, or not; in the order they are written in, since the compiler
// would have all addresses of a state in registers at a time.
__device__ __forceinline__ float load_if(bool there, const float *from)
{
    float r;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %2, 0;\n\t"
                 "mov.b32 %0, 0;\n\t"
                 "@p ld.global.b32 %0, [%1];\n\t}"
                 : "=f"(r)
                 : "l"(from), "r"(static_cast<int>(there))
                 : "memory");
    return r;
}
__device__ __forceinline__ void store_if(bool there, float *to, float v)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %2, 0;\n\t"
                 "@p st.global.b32 [%0], %1;\n\t}" ::"l"(to),
                 "f"(v), "r"(static_cast<int>(there))
                 : "memory");
}

// ---- the kernel ------------------------------------------------------------------------------
// Thread layout, in warpgroups: two of scores' warps (whose spare places take the two issuing
// warps, the decays' warp and the one that asks for copies), the output warps, the state warps,
// and the loaders, who with TMA have nothing to load and write w v in the state warps' stead.
template <int KP, bool TMA>
struct Warps {
    static constexpr int kOutIssue = 2, kStateIssue = 3, kDecay = 6, kCopy = 7;
    static constexpr int kOut = 8;
    static constexpr int kState = 12, kStates = 4 * (KP / 64);
    static constexpr int kLoad = kState + kStates;
    static constexpr int kThreads = kLoad * 32 + kLoaders;
    static constexpr int kWeighers = TMA ? kLoaders : kStates * 32;  // who write w v
};
// Tensor memory: two buffers of scores (intra goes where its scores were), one or two of
// inter, the update, and S^T in up to three parts.
template <typename T, int KP>
struct Columns {
    static constexpr int kInters = KP + Parts<T>::kMid * KP / 2 <= 256 ? 2 : 1;
    static constexpr int kScores = 0, kInter = 128, kUpdate = kInter + kInters * C,
                         kState = kUpdate + KP;
    static_assert(kState + Parts<T>::kMid * KP / 2 <= 512, "tensor memory");
};

// Conditions that keep their code out of the way.
__device__ __forceinline__ bool rare(bool c) { return __builtin_expect(c, 0); }

// D = the products of parts that matter, over `steps` blocks of 16 along the sum (one more
// where they are odd: the operands are zeros there); a, b: an operand's descriptor for a part
// and a block.  One thread of the warp issues; it does so in a branch that the compiler knows
// to be one thread's, else every descriptor costs ten instructions.
template <int NA, int NB, typename A, typename B, typename M>
__device__ __forceinline__ void multiply(bool leader, int steps, const A &a, const B &b, const M &mma,
                                         bool more = false)
{
    constexpr int most = NA > NB ? NA : NB;
    if (leader) {
        // the small products first
#pragma unroll 1
        for (int order = most - 1; order >= 0; --order)
#pragma unroll 1
            for (int i = order < NB ? 0 : order - NB + 1; i < NA && i <= order; ++i)
#pragma unroll 1
                for (int k = 0; k < steps; k += 2) {
#pragma unroll
                    for (int m = 0; m < 2; ++m)
                        mma(a(i, k + m), b(order - i, k + m), more || m > 0);
                    more = true;
                }
    }
}

template <typename T, int KP, bool TMA>
__global__ void __launch_bounds__(Warps<KP, TMA>::kThreads, 1)
attention_kernel(const __grid_constant__ Maps maps, const AttentionArgs p, const Spans spans,
                 const bool outputs, const bool ordered, const Layout l, const int aligned,
                 unsigned *fault, const KernelTest test)
{
    using W = Warps<KP, TMA>;
    using Col = Columns<T, KP>;
    using P = Parts<T>;
    constexpr int kWeighers = W::kWeighers;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *const weighted = smem + l.stages * l.stage;
    uint8_t *const p_tiles = weighted + l.weighted;
    uint8_t *const staging = p_tiles + l.p_buffers * l.p;
    Decays *const decays = reinterpret_cast<Decays *>(staging + l.staging);
    Info *const infos = reinterpret_cast<Info *>(decays + kMaxStages);
    Barriers &bar = *reinterpret_cast<Barriers *>(infos + kInfos);
    volatile int *const abort = &bar.abort;

    if (!outputs)
        ptx::griddep_launch_dependents();  // (the joining)
    ptx::griddep_wait();
    // (the same for a warp's lanes, and known to be)
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int v0 = blockIdx.z * 128, values = min(p.values - v0, 128);
    int head = blockIdx.y, sequence = blockIdx.x, number = 0;
    if (spans.tokens) {
        sequence = tile_owner(p.seq, blockIdx.x, spans.tokens, &number);
    } else if (ordered) {
        // the longest sequences' heads go first, so that no long one starts when the others end
        // (the grid is heads x sequences then)
        head = blockIdx.x;
        int *const lengths = reinterpret_cast<int *>(smem);
        const int n = threadIdx.x, count = p.seq.count;
        const int own = n < count ? sequence_end(p.seq, n) - sequence_begin(p.seq, n) : -1;
        if (n < kOrdered)
            lengths[n] = own;
        __syncthreads();
        if (n < count) {
            int rank = 0;
#pragma unroll 2
            for (int m = 0; m < count; m += 4) {
                const int4 some = *reinterpret_cast<const int4 *>(lengths + m);
                const int others[4] = {some.x, some.y, some.z, some.w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    rank += others[k] > own || (others[k] == own && m + k < n);
            }
            if (rank == static_cast<int>(blockIdx.y))
                bar.sequence = n;
        }
        __syncthreads();
        sequence = __shfl_sync(0xffffffffu, bar.sequence, 0);
    }
    const int slot = sequence_slot(p.slots, sequence);
    Run run;
    run.begin = sequence_begin(p.seq, sequence);
    run.end = sequence_end(p.seq, sequence);
    run.to = slot >= 0 ? p.state_of(slot, head) + v0 : nullptr;
    run.from = run.to && sequence_resumes(p.slots, sequence) ? run.to : nullptr;
    if (spans.tokens) {
        const int count = spans.count(run.end - run.begin);
        // (a few numbers own no rows, those before the first sequence's are negative; what the last
        // span leaves is made with its outputs)
        if (number < 0 || number >= count || (!outputs && number == count - 1))
            return;
        if (!outputs) {
            run.from = nullptr;
            run.to = spans.state_of(p, blockIdx.x + 1, head) + v0;
        } else if (count > 1) {
            if (number > 0 || run.from)
                run.from = spans.state_of(p, blockIdx.x, head) + v0;
            if (number < count - 1)
                run.to = nullptr;
        }
        run.begin += number * spans.tokens;
        run.end = min(run.end - run.begin, spans.tokens) + run.begin;
    }
    const int chunks = (run.end - run.begin + C - 1) / C;

    // (what lies above P's diagonal stays zero, and so do columns behind keys and values)
    const auto clear = [&](uint8_t *at, int bytes) {
        for (int n = threadIdx.x; n < bytes / 16; n += W::kThreads)
            reinterpret_cast<uint4 *>(at)[n] = make_uint4(0, 0, 0, 0);
    };
    clear(p_tiles, l.p_buffers * l.p);
    if (!TMA)
        clear(smem, min(l.stages, chunks) * l.stage);
    ptx::fence_proxy_async_smem();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            ptx::mbar_init(&bar.full[s], TMA ? 2 : kLoaders / 32 + 1);
            ptx::mbar_init(&bar.empty[s], outputs ? 2 : 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(&bar.scores_full[b], 1);
            ptx::mbar_init(&bar.p_full[b], 3);
            ptx::mbar_init(&bar.inter_full[b], 1);
            ptx::mbar_init(&bar.intra_full[b], 1);
            ptx::mbar_init(&bar.y_free[b], 4);
            ptx::mbar_init(&bar.weighted_full[b], kWeighers / 32);
            ptx::mbar_init(&bar.weighted_free[b], 1);
            ptx::mbar_init(&bar.done[b], 1);
        }
        for (int b = 0; b < kCleans; ++b)
            ptx::mbar_init(&bar.clean[b], kWeighers / 32);
        ptx::mbar_init(&bar.state_full, W::kStates);
        ptx::mbar_init(&bar.update_free, W::kStates);
        ptx::mbar_init(&bar.update_full, 1);
        bar.abort = 0;
        ptx::fence_mbar_init();
    }
    if (warp == W::kOutIssue) {
        ptx::tmem_alloc(&bar.tmem, 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, bar.tmem, 0);
    // the stage of the next chunk, and the parity of its turn
    const auto advance = [&](int &s, uint32_t &turn) {
        if (++s == l.stages) {
            s = 0;
            turn ^= 1;
        }
    };
    // where a chunk stands in buffers used in turn
    const auto parity_of = [](int c, uint32_t buffers) { return static_cast<uint32_t>(c) / buffers & 1; };
    // By all lanes of a warp.  A wait that runs out leaves a mark, and this thread's further
    // waits give up at once: its loops go on to their ends, which takes no code, over whatever
    // the buffers hold.
    unsigned polls = static_cast<unsigned>(test.wait_limit_ns / ptx::kSuspendedNs) + 2;
    const auto wait = [&](uint64_t *b, uint32_t parity, unsigned code) {
        if (!ptx::mbar_wait_suspended(b, parity, polls)) {
            polls = 1;
            *abort = code;
        }
        __syncwarp();
    };
    // what all lanes did before is there
    const auto arrive = [&](uint64_t *b) {
        __syncwarp();
        if (lane == 0)
            ptx::mbar_arrive(b);
    };
    // w v of chunk c in two halves, and V's tile without what the products must not meet
    const auto weigh = [&](int c, int s, uint32_t turn, int tid) {
        wait(&bar.full[s], turn, kFaultConverter);
        uint8_t *const tile = smem + s * l.stage + P::kIn * 2 * l.tile_k;
        const Decays &d = decays[s];
        int *const first_bad = infos[c & (kInfos - 1)].first_bad;
        const int len = TMA ? min(run.end - run.begin - c * C, C) : C;
        if (TMA && rare(len < C)) {
            // rows of other tokens came along: none of their keys joins the state
#pragma unroll 1
            for (int n = tid; n < l.tile_k / 16; n += kWeighers)
                if ((n >> 3 & (C - 1)) >= len)
                    reinterpret_cast<uint4 *>(tile - l.tile_k)[n] = make_uint4(0, 0, 0, 0);
        }
        // A thread takes its units of a half and a slab at a time, rows kRows apart.  Warps of
        // their own write a half when that of the chunk before has been multiplied; the states'
        // warps know that both have been, since they have added the update.
        constexpr bool kOwn = TMA;
        constexpr int kHalf = kSlab / 2, kRows = kWeighers / 8, kTurns = 32 / kRows;
        const int part = l.slabs * kHalf;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
            if (kOwn && c > 0)
                wait(&bar.weighted_free[half], (c - 1) & 1, kFaultConverter);
            const int j0 = half * 32 + (tid >> 3);
            float until[kTurns];
#pragma unroll
            for (int t = 0; t < kTurns; ++t)
                until[t] = d.until[j0 + t * kRows];
#pragma unroll 1
            for (int slab = 0; slab < l.slabs; ++slab) {
                uint8_t *const from = tile + slab * kSlab + half * kHalf + tid * 16;
                uint8_t *const to = weighted + half * (l.weighted / 2) + slab * kHalf + tid * 16;
                Pair f[kTurns][4], none = make_pair(0.0f, 0.0f);
#pragma unroll
                for (int t = 0; t < kTurns; ++t) {
                    load_parts<P::kIn>(from + t * kRows * kRowBytes, l.tile_v, f[t]);
                    if (TMA && rare(j0 + t * kRows >= len)) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            f[t][i] = make_pair(0.0f, 0.0f);
                        *reinterpret_cast<uint4 *>(from + t * kRows * kRowBytes) = make_uint4(0, 0, 0, 0);
                    }
                }
#pragma unroll
                for (int t = 0; t < kTurns; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        none = free_fma2(f[t][i], make_pair(0.0f, 0.0f), none);
                        f[t][i] = free_mul2(f[t][i], make_pair(until[t], until[t]));
                    }
#pragma unroll
                for (int t = 0; t < kTurns; ++t)
                    store_three<(P::kIn > 1)>(to + t * kRows * kRowBytes, part, f[t]);
                const float2 any = split_pair(none);
                if (rare(any.x != 0.0f || any.y != 0.0f)) {
#pragma unroll 1
                    for (int t = 0; t < kTurns; ++t)
                        not_finite<P::kIn>(from + t * kRows * kRowBytes, l.tile_v,
                                           first_bad + slab * 64 + ((tid ^ j0) & 7) * 8,
                                           j0 + t * kRows);
                }
            }
            ptx::fence_proxy_async_smem();
            arrive(&bar.weighted_full[half]);
        }
        if (lane == 0)
            ptx::mbar_arrive(&bar.clean[c & (kCleans - 1)]);
    };

    if (warp < W::kOut && (warp & 3) < 2) {
        // ---- scores to P: lanes are queries; a warp takes 32 of them and 32 keys ----
        const int quarter = warp & 3, half = warp >> 2, i = quarter * 32 + lane;
        if (outputs && half <= quarter) {  // (keys behind all of the queries: zeros)
            int s = 0;
            uint32_t turn = 0;
            for (int c = 0; c < chunks; ++c, advance(s, turn)) {
                const int b = c & 1;
                const uint32_t columns = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                                         Col::kScores + C * b + 32 * half;
                const Decays &d = decays[s];
                // (P of an earlier chunk in this buffer has been multiplied)
                const int before = c - l.p_buffers;
                if (before >= 0)
                    wait(&bar.intra_full[before & 1], parity_of(before, 2), kFaultConverter);
                wait(&bar.full[s], turn, kFaultConverter);
                wait(&bar.scores_full[b], parity_of(c, 2), kFaultConverter);
                ptx::tc_fence_after();
                uint8_t *const row = p_tiles + (c & (l.p_buffers - 1)) * l.p + i * kRowBytes;
                const int swizzle = (i & 7) << 4;
                const Pair mine = *reinterpret_cast<const Pair *>(&d.sum[i]);
                const Pair minus = make_pair(-1.0f, -1.0f);
#pragma unroll 1
                for (int j0 = 0; j0 < 32; j0 += 16) {
                    uint32_t r[16];
                    ptx::tmem_ld_32x32b_x16(columns + j0, r);
                    ptx::tmem_ld_wait();
                    const int at = half * 32 + j0;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float f[8];
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            const int j = u * 8 + e;
                            const ulonglong2 other =
                                *reinterpret_cast<const ulonglong2 *>(&d.sum[at + j]);
                            const float2 one = split_pair(free_fma2(other.x, minus, mine));
                            const float2 two = split_pair(free_fma2(other.y, minus, mine));
                            f[e] = j <= i - at ? __uint_as_float(r[j]) * ex2(one.x + one.y) : 0.0f;
                            f[e + 1] = j + 1 <= i - at ? __uint_as_float(r[j + 1]) * ex2(two.x + two.y)
                                                       : 0.0f;
                        }
                        store_parts<P::kMid>(row + (((at / 8 + u) << 4) ^ swizzle), kSlab, f);
                    }
                }
                ptx::fence_proxy_async_smem();
                ptx::tc_fence_before();
                arrive(&bar.p_full[b]);
            }
        }
    } else if (warp >= W::kOut && warp < W::kState) {
        // ---- inter and intra to y: lanes are values ----
        const int quarter = warp & 3, v = quarter * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        T *const first = p.out<T>(run.begin, head) + v0 + quarter * 32;
        T *const slice = reinterpret_cast<T *>(staging) + quarter * (kOutRows<KP> * 32);
        const int width = values - quarter * 32;  // of this warp's values
        const Pair scale = make_pair(p.scale, p.scale);
        // tokens from `begin` on of a chunk of `len`, whose y is in the slice
        const auto store = [&](T *at, int begin, int len) {
            __syncwarp();
            T *const to = at + begin * p.y_stride;
            const int rows = min(len - begin, kOutRows<KP>);
            if (aligned & 8) {
                // 8 values of 8 rows at a time
                const int col = (lane & 3) * 8;
#pragma unroll 1
                for (int e0 = lane >> 2; e0 < rows; e0 += 32) {
                    Pack<T, 8> some[4];
#pragma unroll
                    for (int n = 0; n < 4; ++n)
                        some[n] = *reinterpret_cast<const Pack<T, 8> *>(slice + (e0 + n * 8) * 32 + col);
#pragma unroll
                    for (int n = 0; n < 4; ++n)
                        if (e0 + n * 8 < rows && col < width)
                            store_pack<T, 8>(to + (e0 + n * 8) * p.y_stride + col, some[n]);
                }
            } else if (lane < width) {
#pragma unroll 1
                for (int e = 0; e < rows; ++e)
                    to[e * p.y_stride + lane] = slice[e * 32 + lane];
            }
            __syncwarp();
        };
        for (int c = 0; outputs && c < chunks; ++c) {
            const int b = c & 1, ib = c & (Col::kInters - 1);
            wait(&bar.inter_full[ib], parity_of(c, Col::kInters), kFaultEpilogue);
            wait(&bar.intra_full[b], parity_of(c, 2), kFaultEpilogue);
            ptx::tc_fence_after();
            const int len = min(run.end - run.begin - c * C, C);
            const Info &info = infos[c & (kInfos - 1)];
            T *const at = first + static_cast<long long>(c) * C * p.y_stride;
            if (width > 0) {
                // the first token that has a value in this column which is not finite
                const int bad = info.first_bad[v];
                const bool all_good = __all_sync(0xffffffffu, bad >= C);
                const uint32_t columns = tmem + lanes + Col::kScores + C * b;
                const uint32_t inter = tmem + lanes + Col::kInter + C * ib;
                T *out = at + lane;
#pragma unroll 1
                for (int e0 = 0; e0 < C; e0 += 16) {
                    uint32_t r[16], past[16];
                    ptx::tmem_ld_32x32b_x16(columns + e0, r);
                    ptx::tmem_ld_32x32b_x16(inter + e0, past);
                    ptx::tmem_ld_wait();
                    float f[16];
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const ulonglong2 since = *reinterpret_cast<const ulonglong2 *>(&info.since[e0 + e]);
#pragma unroll
                        for (int n = 0; n < 4; n += 2) {
                            const float2 two = split_pair(free_mul2(
                                scale, free_fma2(make_pair(__uint_as_float(past[e + n]),
                                                      __uint_as_float(past[e + n + 1])),
                                            n == 0 ? since.x : since.y,
                                            make_pair(__uint_as_float(r[e + n]),
                                                      __uint_as_float(r[e + n + 1])))));
                            f[e + n] = two.x;
                            f[e + n + 1] = two.y;
                        }
                    }
                    if (rare(!all_good)) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            f[e] = e0 + e >= bad ? __uint_as_float(0x7fffffffu) : f[e];
                    }
                    if constexpr (sizeof(T) == 2) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            slice[((e0 & (kOutRows<KP> - 1)) + e) * 32 + lane] = Elem<T>::put(f[e]);
                        if (kOutRows<KP> < C && (e0 & 16))
                            store(at, e0 - 16, len);
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            if (lane < width && e0 + e < len)
                                *out = Elem<T>::put(f[e]);
                            out += p.y_stride;
                        }
                    }
                }
            }
            ptx::tc_fence_before();
            arrive(&bar.y_free[b]);
            if (sizeof(T) == 2 && kOutRows<KP> == C)
                store(at, 0, len);
        }
    } else if (warp >= W::kState && warp < W::kLoad) {
        // ---- states: w v, S, and S as an operand ----
        const int quarter = warp & 3, k0 = ((warp - W::kState) >> 2) * 64;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const int v = quarter * 32 + lane, tid = threadIdx.x - W::kState * 32;
        const bool inside = v < values;
        Pair h[32];  // pairs of keys
        const int some = inside ? p.keys - k0 : 0;  // keys of this lane's h
        {
            const float *from = run.from + k0 * p.values + v;
            const int there = run.from ? some : 0;
#pragma unroll
            for (int n = 0; n < 64; n += 2) {
                const float one = load_if(n < there, from);
                from += p.values;
                h[n / 2] = make_pair(one, load_if(n + 1 < there, from));
                from += p.values;
            }
        }
        int s = 0;
        uint32_t turn = 0;
        // chunk c: its update joins the state; then w v of the next one, and the state for it
#pragma unroll 1
        for (int c = -1; c < chunks; ++c) {
            if (c >= 0) {
                wait(&bar.update_full, c & 1, kFaultConverter);
                ptx::tc_fence_after();
                const float all = infos[c & (kInfos - 1)].all;
                const Pair left = make_pair(all, all);
#pragma unroll
                for (int n0 = 0; n0 < 64; n0 += 8) {
                    uint32_t r[8];
                    ptx::tmem_ld_32x32b_x8(tmem + lanes + Col::kUpdate + k0 + n0, r);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int n = 0; n < 8; n += 2)
                        h[(n0 + n) / 2] = free_fma2(h[(n0 + n) / 2], left,
                                               make_pair(__uint_as_float(r[n]), __uint_as_float(r[n + 1])));
                }
                ptx::tc_fence_before();
                arrive(&bar.update_free);
            }
            if (c + 1 == chunks)
                break;
            if (!TMA) {
                weigh(c + 1, s, turn, tid);
                advance(s, turn);
            }
            if (!outputs)
                continue;
            if (c >= 0) {
                // S of chunk c has been multiplied
                wait(&bar.inter_full[c & (Col::kInters - 1)], parity_of(c, Col::kInters), kFaultConverter);
                ptx::tc_fence_after();
            }
#pragma unroll
            for (int n0 = 0; n0 < 32; n0 += 8) {
                uint32_t r[P::kMid][8];
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    uint32_t parts[P::kMid];
                    const float2 two = split_pair(h[n0 + n]);
                    split_pair_parts<P::kMid>(two.x, two.y, parts);
#pragma unroll
                    for (int part = 0; part < P::kMid; ++part)
                        r[part][n] = parts[part];
                }
#pragma unroll
                for (int part = 0; part < P::kMid; ++part)
                    ptx::tmem_st_32x32b_x8(
                        tmem + lanes + Col::kState + part * (KP / 2) + k0 / 2 + n0, r[part]);
            }
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            arrive(&bar.state_full);
        }
        if (run.to && !*abort) {
            float *to = run.to + k0 * p.values + v;
#pragma unroll
            for (int n = 0; n < 64; ++n) {
                const float2 two = split_pair(h[n / 2]);
                store_if(n < some, to, n % 2 ? two.y : two.x);
                to += p.values;
            }
        }
    } else if (warp == W::kOutIssue) {
        // ---- the outputs' products ----
        const bool leader = ptx::elect_one();
        if (outputs) {
            constexpr uint32_t idesc = ptx::f16_idesc(128, C, true);
            constexpr uint32_t idesc_v = ptx::f16_idesc(128, C, true, true, false);
            const int steps = (p.keys + 15) / 16;
            // descriptors count 16 bytes: a part or a block further is a number added
            const uint64_t p_descs = ptx::sw128_desc(ptx::smem_u32(p_tiles));
            const int part_k = l.tile_k >> 4, part_v = l.tile_v >> 4;
            const auto along_keys = [&](uint64_t desc, int part, int k) {
                return desc + part * part_k + (k >> 2) * (kSlab >> 4) + (k & 3) * 2;
            };
            // scores, intra of the chunk before (with one stage, whose tiles the next scores
            // want gone: of the same chunk), inter
            const int lag = l.stages > 1 ? 1 : 0;
            int s = 0, s_intra = 0;
            uint32_t turn = 0;
#pragma unroll 1
            for (int c = 0; c < chunks + lag; ++c) {
                uint8_t *const stage = smem + s * l.stage;
                const uint64_t q_desc = ptx::sw128_desc(ptx::smem_u32(stage));
                if (c < chunks) {
                    // a buffer of scores is free, and so is one of two of inter, when y of the
                    // chunk before in it has been read
                    wait(&bar.full[s], turn, kFaultMma);
                    if (c >= 2)
                        wait(&bar.y_free[c & 1], parity_of(c - 2, 2), kFaultMma);
                    ptx::tc_fence_after();
                    const uint64_t k_desc = q_desc + P::kIn * part_k;
                    const uint32_t scores = tmem + Col::kScores + C * (c & 1);
                    multiply<P::kIn, P::kIn>(
                        leader, steps, [&](int i, int k) { return along_keys(q_desc, i, k); },
                        [&](int j, int k) { return along_keys(k_desc, j, k); },
                        [&](uint64_t a, uint64_t b_desc, bool more) {
                            ptx::mma_f16(scores, a, b_desc, idesc, more);
                        });
                    if (leader)
                        ptx::mma_commit(&bar.scores_full[c & 1]);
                }
                const int of = c - lag;
                if (of >= 0) {
                    // (w v is there: what is not finite has left V's tile)
                    wait(&bar.p_full[of & 1], parity_of(of, 2), kFaultMma);
                    wait(&bar.clean[of & (kCleans - 1)], parity_of(of, kCleans), kFaultMma);
                    ptx::tc_fence_after();
                    const uint64_t p_desc = p_descs + (of & (l.p_buffers - 1)) * (l.p >> 4);
                    const uint64_t v_desc = ptx::sw128_desc(
                        ptx::smem_u32(smem + s_intra * l.stage + P::kIn * 2 * l.tile_k), kSlab);
                    const uint32_t intra = tmem + Col::kScores + C * (of & 1);
                    multiply<P::kIn, P::kMid>(
                        leader, C / 16,
                        [&](int i, int k) { return v_desc + i * part_v + k * (2048 >> 4); },
                        [&](int j, int k) { return p_desc + j * (kSlab >> 4) + k * 2; },
                        [&](uint64_t a, uint64_t b_desc, bool more) {
                            ptx::mma_f16(intra, a, b_desc, idesc_v, more);
                        });
                    if (leader) {
                        ptx::mma_commit(&bar.intra_full[of & 1]);
                        if (lag)
                            ptx::mma_commit(&bar.empty[s_intra]);
                    }
                }
                s_intra = s;
                if (c < chunks) {
                    wait(&bar.state_full, c & 1, kFaultMma);
                    if (Col::kInters == 1 && c > 0)
                        wait(&bar.y_free[(c - 1) & 1], parity_of(c - 1, 2), kFaultMma);
                    ptx::tc_fence_after();
                    const uint32_t inter = tmem + Col::kInter + C * (c & (Col::kInters - 1));
                    multiply<P::kMid, P::kIn>(
                        leader, steps,
                        [&](int i, int k) { return tmem + Col::kState + i * (KP / 2) + k * 8; },
                        [&](int j, int k) { return along_keys(q_desc, j, k); },
                        [&](uint32_t a, uint64_t b_desc, bool more) {
                            ptx::mma_f16_tmem_a(inter, a, b_desc, idesc, more);
                        });
                    if (leader) {
                        ptx::mma_commit(&bar.inter_full[c & (Col::kInters - 1)]);
                        if (!lag)
                            ptx::mma_commit(&bar.empty[s]);
                    }
                }
                advance(s, turn);
            }
            // every product has completed before tensor memory is freed
            if (leader)
                ptx::mma_commit(&bar.done[0]);
            __syncwarp();
            ptx::mbar_wait_drain(&bar.done[0], 0, fault, kDefaultWaitLimitNs);
        }
    } else if (warp == W::kStateIssue) {
        // ---- the states' products ----
        {
            const bool leader = ptx::elect_one();
            constexpr uint32_t idesc = ptx::f16_idesc(128, KP, true, true, true);
            const int part_w = l.slabs * (kSlab / 2) >> 4;
            int s = 0;
            uint32_t turn = 0;
#pragma unroll 1
            for (int c = 0; c < chunks; ++c, advance(s, turn)) {
                wait(&bar.full[s], turn, kFaultMma);
                if (c > 0)
                    wait(&bar.update_free, (c - 1) & 1, kFaultMma);
                const uint64_t k_desc = ptx::sw128_desc(
                    ptx::smem_u32(smem + s * l.stage) + P::kIn * l.tile_k, kSlab);
                const uint64_t w_desc = ptx::sw128_desc(ptx::smem_u32(weighted), kSlab / 2);
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    wait(&bar.weighted_full[half], c & 1, kFaultMma);
                    ptx::tc_fence_after();
                    const uint64_t a_desc = w_desc + half * (l.weighted >> 5);
                    const uint64_t b_desc = k_desc + half * (kSlab >> 5);
                    multiply<kWeighted, P::kIn>(
                        leader, C / 32, [&](int i, int k) { return a_desc + i * part_w + k * (2048 >> 4); },
                        [&](int j, int k) { return b_desc + j * (l.tile_k >> 4) + k * (2048 >> 4); },
                        [&](uint64_t a, uint64_t b, bool more) {
                            ptx::mma_f16(tmem + Col::kUpdate, a, b, idesc, more);
                        },
                        half > 0);
                    if (leader) {
                        ptx::mma_commit(&bar.weighted_free[half]);
                        if (half == 1) {
                            ptx::mma_commit(&bar.update_full);
                            ptx::mma_commit(&bar.empty[s]);
                        }
                    }
                }
            }
            if (leader)
                ptx::mma_commit(&bar.done[1]);
            __syncwarp();
            ptx::mbar_wait_drain(&bar.done[1], 0, fault, kDefaultWaitLimitNs);
        }
    } else if (warp == W::kDecay) {
        const auto decay_at = [&](int c, int i) {
            const int t = run.begin + c * C + i;
            return t < run.end ? __ldg(p.decay + t * p.decay_stride + head) : 0.0f;
        };
        float g0 = decay_at(0, 2 * lane), g1 = decay_at(0, 2 * lane + 1);
        Sum total = {0.0f, 0.0f};
        int s = 0;
        uint32_t turn = 0;
        for (int c = 0; c < chunks; ++c, advance(s, turn)) {
            const float n0 = decay_at(c + 1, 2 * lane), n1 = decay_at(c + 1, 2 * lane + 1);
            if (c >= l.stages)
                wait(&bar.empty[s], turn ^ 1, kFaultProducer);
            total = add(total, sum_decays(decays[s], infos[c & (kInfos - 1)], g0, g1, lane));
            arrive(&bar.full[s]);
            g0 = n0;
            g1 = n1;
        }
        if (!outputs && lane == 0 && blockIdx.z == 0)
            *spans.left_of(p, blockIdx.x, head) = ex2(total.hi + total.lo);
    } else if (TMA && warp == W::kCopy && !test.withhold) {
        // ---- rows by TMA (failure test: nothing is loaded, so the waits for it run out) ----
        const int q_head = head / p.q.share, k_head = head / p.k.share, v_head = head / p.v.share;
        const uint32_t bytes = (outputs ? 2 : 1) * l.tile_k + l.tile_v;
        int s = 0, c = 0;
        uint32_t turn = 0;
        for (; c < chunks; ++c, advance(s, turn)) {
            if (c >= l.stages)
                wait(&bar.empty[s], turn ^ 1, kFaultProducer);
            if (polls == 1)  // (nothing is copied over what may be on its way)
                break;
            if (lane == 0) {
                uint64_t *const full = &bar.full[s];
                uint8_t *const to = smem + s * l.stage;
                const int t0 = run.begin + c * C;
                ptx::mbar_arrive_expect_tx(full, bytes);
#pragma unroll
                for (int slab = 0; slab < KP / 64; ++slab) {
                    if (outputs)
                        ptx::tma_load_3d(to + slab * kSlab, &maps.of[0], full, slab * 64, q_head, t0);
                    ptx::tma_load_3d(to + l.tile_k + slab * kSlab, &maps.of[1], full, slab * 64, k_head, t0);
                }
#pragma unroll
                for (int slab = 0; slab < 2; ++slab)
                    if (slab < l.slabs)
                        ptx::tma_load_3d(to + 2 * l.tile_k + slab * kSlab, &maps.of[2], full,
                                         v0 + slab * 64, v_head, t0);
            }
        }
        // every load has landed before the CTA's shared memory goes away
        for (int n = max(c - l.stages, 0); n < c; ++n)
            ptx::mbar_wait_drain(&bar.full[n % l.stages], n / l.stages & 1, fault, kDefaultWaitLimitNs);
    } else if (TMA && warp >= W::kLoad) {
        // ---- w v ----
        int s = 0;
        uint32_t turn = 0;
        for (int c = 0; c < chunks; ++c, advance(s, turn))
            weigh(c, s, turn, threadIdx.x - W::kLoad * 32);
    } else if (warp >= W::kLoad && !test.withhold) {
        // ---- loaders: a group of rows is read while the one before is written ----
        const int tid = threadIdx.x - W::kLoad * 32, first = outputs ? 0 : 1;
        const auto width_of = [&](int which) { return which == 2 ? values : p.keys; };
        const auto units_of = [&](int which) { return 32 - __clz((width_of(which) + 7) / 8 - 1); };
        int s = 0, c = 0, which = first, group = 0;
        uint32_t turn = 0;
        const auto read = [&](float (&f)[kTogether][8]) {
            const HeadRows &m = which == 0 ? p.q : which == 1 ? p.k : p.v;
            const T *const from = m.row<T>(run.begin + static_cast<long long>(c) * C, head) +
                                  (which == 2 ? v0 : 0);
            const int len = run.end - run.begin - c * C, width = width_of(which);
            // the next chunk's rows are on their way to L2 meanwhile, two threads a row
            const int row = C + (tid >> 1);
            if (group == 0 && row < len) {
                const char *next = reinterpret_cast<const char *>(from + row * m.stride);
#pragma unroll 1
                for (int n = (tid & 1) * 128; n < width * static_cast<int>(sizeof(T)); n += 256)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(next + n));
            }
            read_rows<T>(f, from, m.stride, aligned >> which & 1, len, width, units_of(which), group, tid);
        };
        // false: there is no further group
        const auto step = [&](const float (&f)[kTogether][8], float (&next)[kTogether][8]) {
            const int c0 = c, which0 = which, group0 = group;
            const int units = units_of(which);
            if (++group >= 1 << units >> 2) {
                group = 0;
                if (++which == 3) {
                    which = first;
                    ++c;
                }
            }
            if (c < chunks)
                read(next);
            if (which0 == first && group0 == 0 && c0 >= l.stages)
                wait(&bar.empty[s], turn ^ 1, kFaultProducer);
            write_rows<P::kIn>(f, smem + s * l.stage + which0 * P::kIn * l.tile_k,
                               which0 == 2 ? l.tile_v : l.tile_k, units, group0, tid);
            if (c > c0) {
                ptx::fence_proxy_async_smem();
                arrive(&bar.full[s]);
                advance(s, turn);
            }
            return c < chunks;
        };
        if (chunks > 0) {
            float now[kTogether][8], next[kTogether][8];
            read(now);
#pragma unroll 1
            while (step(now, next)) {
#pragma unroll
                for (int k = 0; k < kTogether; ++k)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        now[k][j] = next[k][j];
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort)
        atomicOr(fault, static_cast<unsigned>(*abort));
    if (warp == W::kOutIssue) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

template <typename T, int KP, bool TMA>
int launch(const Maps &maps, int aligned, const AttentionArgs &p, const Spans &spans, bool outputs,
           cudaStream_t stream)
{
    using W = Warps<KP, TMA>;
    static SharedMemory memory;
    const Layout l = layout<T, KP>(p.values < 128 ? p.values : 128);
    int st = memory.allow(attention_kernel<T, KP, TMA>, 227 * 1024);
    if (st != LSTM_OK)
        return st;
    unsigned *fault = fault_word();
    if (!fault)
        return fail(LSTM_E_CUDA, "cannot resolve the device fault word");
    if ((st = check_launch_injection("lstm_linear_attention")))
        return st;
    const bool ordered = !spans.tokens && p.seq.offsets && p.seq.count > 1 && p.seq.count <= kOrdered;
    const unsigned units = static_cast<unsigned>(spans.tokens ? spans.units : p.seq.count),
                   heads = static_cast<unsigned>(p.heads);
    const dim3 grid(ordered ? heads : units, ordered ? units : heads,
                    static_cast<unsigned>((p.values + 127) / 128));
    Dependent launch(grid, W::kThreads, l.total, stream);
    if (!(spans.tokens && outputs))  // nothing of this call comes before
        launch.config.numAttrs = 0;
    return cuda_status(cudaLaunchKernelEx(&launch.config, attention_kernel<T, KP, TMA>, maps, p, spans,
                                          outputs, ordered, l, aligned, fault,
                                          kernel_test(kTestAttention)),
                       "lstm_linear_attention launch");
}

template <typename T, int KP, bool TMA>
int launch_passes(const Maps &maps, int aligned, const AttentionArgs &p, const Spans &spans,
                  cudaStream_t stream)
{
    int st;
    if (spans.tokens && ((st = launch<T, KP, TMA>(maps, aligned, p, spans, false, stream)) ||
                         (st = launch_attention_join(p, spans, stream))))
        return st;
    return launch<T, KP, TMA>(maps, aligned, p, spans, true, stream);
}

template <typename T, int KP>
int launch_all(const AttentionArgs &p, const Spans &spans, cudaStream_t stream)
{
    Maps maps = {};
    const int tokens = p.seq.tokens;
    int aligned = 0;
    const auto in_place = [&](const HeadRows &m) {
        return rows_aligned(m.at, tokens > 1 ? m.stride : 0, sizeof(T)) &&
               m.head_stride * sizeof(T) % 16 == 0;
    };
    aligned = in_place(p.q) | in_place(p.k) << 1 | in_place(p.v) << 2;
    if (rows_aligned(p.y, tokens > 1 ? p.y_stride : 0, sizeof(T)) && p.values % 8 == 0)
        aligned |= 8;
    if constexpr (Parts<T>::kIn == 1) {
        // (a map that the driver does not make: the rows are loaded by threads)
        const auto map = [&](CUtensorMap *to, const HeadRows &m, int width) {
            return encode_heads_map(to, m.at, tokens, p.heads / m.share, width, m.stride, m.head_stride);
        };
        if ((aligned & 7) == 7 && tokens > 0 && map(&maps.of[0], p.q, p.keys) &&
            map(&maps.of[1], p.k, p.keys) && map(&maps.of[2], p.v, p.values))
            return launch_passes<T, KP, true>(maps, aligned, p, spans, stream);
    }
    return launch_passes<T, KP, false>(maps, aligned, p, spans, stream);
}

template <typename T>
int launch_keys(const AttentionArgs &p, const Spans &spans, cudaStream_t stream)
{
    return p.keys <= 64 ? launch_all<T, 64>(p, spans, stream) : launch_all<T, 128>(p, spans, stream);
}

}  // namespace prompts
}  // namespace lstm
