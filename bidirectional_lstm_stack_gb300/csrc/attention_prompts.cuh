// Linear attention over prompts, in chunks of 64 tokens on the tensor cores.  With c_i
// the sum of the chunk's log decays up to token i and S the state before it,
//     y_i = scale (e^(c_i) S^T q_i + sum_(j <= i) e^(c_i - c_j) (q_i . k_j) v_j)
//     S'  = e^(c_64) S + sum_j e^(c_64 - c_j) k_j v_j^T.
// A CTA takes one head of one run of tokens and up to 128 of its values, and keeps S
// transposed: tensor-memory lanes are values, so every product has M = 128 lanes and no
// state ever goes through shared memory.  Per chunk the tensor cores make
//     scores   Q K^T            [64 queries x 64 keys]   (lanes are queries)
//     inter    S^T Q^T          [values x 64 queries]    (S^T in tensor memory, bf16)
//     intra    V^T P^T          [values x 64 queries]    (P: decayed, masked scores)
//     update   (wV)^T K         [values x keys]          (w_j = e^(c_64 - c_j))
// and the warps have one task each:
//  * 4 loaders bring q, k and v of the next chunks into a ring of stages (128-byte
//    swizzle, so the same tile serves as K-major and as MN-major operand); a warp beside
//    them sums the log decays, in fp64, since c_i - c_j of far sums would lose what
//    separates near tokens;
//  * 3 warps turn scores into P, 4 others inter and intra into y, a chunk behind;
//  * 4 or 8 state warps hold S in registers (fp32, a lane per value), add the update, write
//    w v of the next chunk and hand S on as bf16;
//  * two threads issue the products, those of the outputs and those of the states, so that
//    neither chain waits for the other.
// Where sequences and heads are fewer than SMs, sequences are cut into spans: a first pass
// makes what each span adds to a state of zeros (no outputs), a small kernel joins them to
// the states that the spans start from, and then all spans run side by side.
// bf16 inputs are exact operands.  P and S are rounded to bf16 for their products (an
// output of bf16 is rounded as coarsely itself); w v goes as three parts of bf16, so that
// what joins the state, which is fp32, keeps 24 bits.  fp16 goes as two parts of bf16
// (exact), so do P and S (which in fp16 itself would overflow); fp32 as three parts
// (exact), and so do P and S.  Of two factors' parts those products are made that the other roundings leave
// visible (parts a, b with a + b below the larger number of parts).
#pragma once

#include "attention.cuh"

namespace lstm {
namespace prompts {

constexpr int C = 64;           // tokens of a chunk
constexpr int kRowBytes = 128;  // of a tile's row: 64 bf16
constexpr int kSlab = C * kRowBytes;
constexpr int kMaxStages = 3;
constexpr int kLoaders = 128;
constexpr float kLeast = -300.0f;  // log2 of a decay that leaves nothing of any fp32 number

// Parts of bf16 that the numbers of a type are split into.
template <typename T>
struct Parts;
template <>
struct Parts<__nv_bfloat16> {
    static constexpr int kIn = 1, kMid = 1;
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

// What one stage holds beside its tiles.
struct Decays {
    float2 sum[C];   // c_i in log2, as the fp32 next to it and the rest
    float until[C];  // e^(c_64 - c_i)
    float all;       // e^(c_64)
    float pad[3];
};

// What the output warps want to know of a chunk, whose stage may be another chunk's by then.
// Chunk c + 5 is loaded when y of chunk c is done at the earliest: three stages, and two
// buffers of scores before y.
struct Info {
    float since[C];      // e^(c_i)
    int first_bad[128];  // of a value's column: the first token that is not finite, or C
};
constexpr int kInfos = 8;
// w v of a chunk is there: the states are two chunks ahead of the outputs at most
constexpr int kWeights = 4;

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
    uint64_t weighted_full[kWeights], state_full, update_full;
    uint64_t done[2];
    uint32_t tmem;
    int abort;
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
    l.staging = sizeof(T) == 2 ? 4 * C * 32 * 2 : 0;
    // (products of 128 lanes read past tiles of 64, into the tile behind them)
    const size_t rest = l.weighted + l.staging + kMaxStages * sizeof(Decays) + kInfos * sizeof(Info) +
                        sizeof(Barriers) + 1024;
    const auto bytes = [&] { return l.stages * l.stage + l.p_buffers * l.p + rest; };
    l.stages = kMaxStages;
    l.p_buffers = 2;
    while (l.stages > 1 && bytes() > 227 * 1024)
        --l.stages;
    if (bytes() > 227 * 1024)
        l.p_buffers = 1;
    l.total = bytes();
    return l;
}

// ---- parts -----------------------------------------------------------------------------
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float low_float(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float high_float(uint32_t pair)
{
    return __uint_as_float(pair & 0xffff0000u);
}
// Two numbers as N pairs of parts: each but the last of three cut off (which leaves the
// rest exact and of no more than 8 bits in the end), those of two rounded to nearest.
template <int N>
__device__ __forceinline__ void split_pair_parts(float x, float y, uint32_t (&r)[N])
{
    if constexpr (N == 3) {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            asm("prmt.b32 %0, %1, %2, 0x7632;" : "=r"(r[k]) : "r"(__float_as_uint(x)), "r"(__float_as_uint(y)));
            x -= low_float(r[k]);
            y -= high_float(r[k]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            r[k] = bf16_pair(x, y);
            if (k + 1 < N) {
                x -= low_float(r[k]);
                y -= high_float(r[k]);
            }
        }
    }
}

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

// The numbers that N units of 16 bytes stand for.
template <int N>
__device__ __forceinline__ void load_parts(const uint8_t *at, int apart, float (&f)[8])
{
#pragma unroll
    for (int k = N - 1; k >= 0; --k) {
        const uint4 u = *reinterpret_cast<const uint4 *>(at + k * apart);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = k == N - 1 ? low_float(w[i]) : f[2 * i] + low_float(w[i]);
            f[2 * i + 1] = k == N - 1 ? high_float(w[i]) : f[2 * i + 1] + high_float(w[i]);
        }
    }
}

// ---- loading ------------------------------------------------------------------------------
// Rows t0 .. t0 + 63 of a head into a tile of `units` 16-byte units a row (8 or 16); rows
// from `len` and numbers from `width` on are zeros.  A thread keeps its unit and goes down
// the rows, so that swizzle and width are worked out once.
template <typename T>
__device__ __forceinline__ void load_tile(uint8_t *tile, int apart, const T *from, long long stride,
                                          bool aligned, int len, int width, int units, int tid)
{
    constexpr int kTogether = 4;              // rows in flight
    const int down = kLoaders / units;        // rows of a turn, a multiple of 8
    const int u = tid & (units - 1), r0 = tid / units;
    const T *src = from + r0 * stride + u * 8;
    const long long step = down * stride;
    uint8_t *dst = tile + (u >> 3) * kSlab + r0 * kRowBytes + (((u & 7) ^ (r0 & 7)) << 4);
    const int there = min(max(width - u * 8, 0), 8);
#pragma unroll 1
    for (int r = r0; r < C; r += kTogether * down) {
        if (Parts<T>::kIn == 1 && aligned) {
#pragma unroll
            for (int k = 0; k < kTogether; ++k) {
                const bool in = r + k * down < len && there > 0;
                // (`from` is an address that may be read, for where there is nothing to read)
                ptx::cp_async_16(ptx::smem_u32(dst + k * down * kRowBytes),
                                 in ? src + k * step : from, in ? there * 2 : 0);
            }
        } else {
            float f[kTogether][8];
            if (aligned && there == 8) {
                constexpr int V = Elem<T>::kVector;
#pragma unroll
                for (int k = 0; k < kTogether; ++k)
#pragma unroll
                    for (int j = 0; j < 8; j += V) {
                        Pack<T, V> v = {};
                        if (r + k * down < len)
                            v = load_pack<T, V>(src + k * step + j);
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            f[k][j + e] = Elem<T>::get(v.v[e]);
                    }
            } else {
#pragma unroll
                for (int k = 0; k < kTogether; ++k)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        f[k][j] = r + k * down < len && j < there ? Elem<T>::get(src[k * step + j])
                                                                  : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < kTogether; ++k)
                store_parts<Parts<T>::kIn>(dst + k * down * kRowBytes, apart, f[k]);
        }
        src += kTogether * step;
        dst += kTogether * down * kRowBytes;
    }
}

// The sums of a chunk's log decays, two tokens a lane; returns the whole sum, in log2.
__device__ __forceinline__ double sum_decays(Decays &d, Info &info, float g0, float g1, int lane)
{
    const auto log2_of = [](float g) {
        const double v = static_cast<double>(g) * 1.4426950408889634;
        return v < kLeast ? static_cast<double>(kLeast) : v;  // (a NaN stays)
    };
    const double a = log2_of(g0), b = log2_of(g1);
    double sum = a + b;
#pragma unroll 1
    for (int m = 1; m < 32; m *= 2) {
        const double other = __shfl_up_sync(0xffffffffu, sum, m);
        if (lane >= m)
            sum += other;
    }
    const double end = __shfl_sync(0xffffffffu, sum, 31);
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        const double c = k ? sum : sum - b;
        const int i = 2 * lane + k;
        const float hi = static_cast<float>(c);
        d.sum[i] = make_float2(hi, static_cast<float>(c - hi));
        d.until[i] = ex2(static_cast<float>(end - c));
        info.since[i] = ex2(hi) * (1.0f + 0.6931472f * static_cast<float>(c - hi));
    }
    *reinterpret_cast<int4 *>(&info.first_bad[4 * lane]) = make_int4(C, C, C, C);
    if (lane == 0)
        d.all = ex2(static_cast<float>(end));
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
        // (of a number that is not finite the first part is neither)
        const unsigned short first = *reinterpret_cast<const unsigned short *>(at);
        if ((first & 0x7f80) == 0x7f80) {
            atomicMin(first_bad + e, j);
#pragma unroll
            for (int k = 0; k < N; ++k)
                *reinterpret_cast<unsigned short *>(at + k * apart) = 0;
        }
    }
}

// ptx::mbar_wait_bounded in as few instructions as it takes: the kernel's warps all run
// different code, and what of it exceeds the instruction cache is fetched for every chunk.
__device__ __forceinline__ bool wait_bounded(uint64_t *bar, uint32_t parity, volatile int *abort,
                                             unsigned *fault, unsigned code, uint64_t limit_ns)
{
    uint64_t start = 0;
#pragma unroll 1
    while (!ptx::mbar_try_wait(bar, parity)) {
        const uint64_t now = ptx::globaltimer();
        if (start == 0)
            start = now;
        if (now - start > limit_ns) {
            atomicOr(fault, code);
            *abort = 1;
        }
        if (*abort)
            return false;
    }
    return true;
}

// ---- the kernel ------------------------------------------------------------------------------
// Thread layout, in warpgroups: two of scores' warps (whose spare places take the two issuing
// warps and the decays' warp), the output warps, the state warps, the loaders.
template <int KP>
struct Warps {
    static constexpr int kOutIssue = 2, kStateIssue = 3, kDecay = 6;
    static constexpr int kOut = 8;
    static constexpr int kState = 12, kStates = 4 * (KP / 64);
    static constexpr int kLoad = kState + kStates;
    static constexpr int kThreads = (kLoad + 4) * 32;
    // Registers: as the block is launched (65536 over its threads), and, with 128 keys, as
    // its warpgroups then share those of the launch
    static constexpr int kRegisters = KP > 64 ? 80 : 96;
    static constexpr bool kShare = KP > 64;
    static constexpr int kScoresRegisters = 72, kOutRegisters = 64, kStateRegisters = 104,
                         kLoadRegisters = 64;
    static_assert(kLoad * 32 + kLoaders == kThreads && kState % 4 == 0, "warpgroups");
    static_assert(!kShare || kThreads * kRegisters == 256 * kScoresRegisters + 128 * kOutRegisters +
                                                          kStates * 32 * kStateRegisters +
                                                          kLoaders * kLoadRegisters,
                  "registers");
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

// D = the products of parts that matter, over `steps` blocks of 16 along the sum (one more
// where they are odd: the operands are zeros there); a, b: an operand's descriptor for a part
// and a block.  One thread of the warp issues; it does so in a branch that the compiler knows
// to be one thread's, else every descriptor costs ten instructions.
template <int NA, int NB, typename A, typename B, typename M>
__device__ __forceinline__ void multiply(bool leader, int steps, const A &a, const B &b, const M &mma)
{
    constexpr int most = NA > NB ? NA : NB;
    if (leader) {
        bool more = false;
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

template <typename T, int KP>
__global__ void __launch_bounds__(Warps<KP>::kThreads, 1)
attention_kernel(const AttentionArgs p, const Spans spans, const bool outputs, const Layout l,
                 const int aligned, unsigned *fault, const KernelTest test)
{
    using W = Warps<KP>;
    using Col = Columns<T, KP>;
    using P = Parts<T>;
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

    // (the same for a warp's lanes, and known to be)
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int head = blockIdx.y, v0 = blockIdx.z * 128;
    const int values = min(p.values - v0, 128);
    int sequence = blockIdx.x, number = 0;
    if (spans.tokens)
        sequence = tile_owner(p.seq, blockIdx.x, spans.tokens, &number);
    const int slot = sequence_slot(p.slots, sequence);
    Run run;
    run.begin = sequence_begin(p.seq, sequence);
    run.end = sequence_end(p.seq, sequence);
    run.to = slot >= 0 ? p.state_of(slot, head) + v0 : nullptr;
    run.from = run.to && sequence_resumes(p.slots, sequence) ? run.to : nullptr;
    if (spans.tokens) {
        const int count = spans.count(run.end - run.begin);
        // (a few numbers own no rows; what the last span leaves is made with its outputs)
        if (number >= count || (!outputs && number == count - 1))
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

    // (what lies above P's diagonal stays zero)
    for (int n = threadIdx.x; n < l.p_buffers * l.p / 16; n += W::kThreads)
        reinterpret_cast<uint4 *>(p_tiles)[n] = make_uint4(0, 0, 0, 0);
    ptx::fence_proxy_async_smem();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            ptx::mbar_init(&bar.full[s], kLoaders + 32);
            ptx::mbar_init(&bar.empty[s], outputs ? 2 : 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(&bar.scores_full[b], 1);
            ptx::mbar_init(&bar.p_full[b], 3 * 32);
            ptx::mbar_init(&bar.inter_full[b], 1);
            ptx::mbar_init(&bar.intra_full[b], 1);
            ptx::mbar_init(&bar.y_free[b], 4 * 32);
            ptx::mbar_init(&bar.done[b], 1);
        }
        for (int b = 0; b < kWeights; ++b)
            ptx::mbar_init(&bar.weighted_full[b], W::kStates * 32);
        ptx::mbar_init(&bar.state_full, W::kStates * 32);
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
    const auto stage_of = [&](int c) { return c % l.stages; };
    const auto turn_of = [&](int c) { return static_cast<uint32_t>(c / l.stages) & 1; };
    // where a chunk stands in buffers used in turn
    const auto parity_of = [](int c, int buffers) { return static_cast<uint32_t>(c / buffers) & 1; };
    // (by all lanes of a warp)
    const auto wait = [&](uint64_t *b, uint32_t parity, unsigned code) {
        return __all_sync(0xffffffffu, wait_bounded(b, parity, abort, fault, code, test.wait_limit_ns)) != 0;
    };

    if constexpr (W::kShare) {
        if (warp < W::kOut)
            ptx::fewer_registers<W::kScoresRegisters>();
        else if (warp < W::kState)
            ptx::fewer_registers<W::kOutRegisters>();
        else if (warp < W::kLoad)
            ptx::more_registers<W::kStateRegisters>();
        else
            ptx::fewer_registers<W::kLoadRegisters>();
    }
    if (warp < W::kOut && (warp & 3) < 2) {
        // ---- scores to P: lanes are queries; a warp takes 32 of them and 32 keys ----
        const int quarter = warp & 3, half = warp >> 2, i = quarter * 32 + lane;
        if (outputs && half <= quarter) {  // (keys behind all of the queries: zeros)
            for (int c = 0; c < chunks; ++c) {
                const int s = stage_of(c), b = c & 1;
                const uint32_t columns = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                                         Col::kScores + C * b + 32 * half;
                const Decays &d = decays[s];
                // (P of an earlier chunk in this buffer has been multiplied)
                const int before = c - l.p_buffers;
                const bool ok = (before < 0 || wait(&bar.intra_full[before & 1],
                                                    parity_of(before, 2), kFaultConverter)) &&
                                wait(&bar.full[s], turn_of(c), kFaultConverter) &&
                                wait(&bar.scores_full[b], parity_of(c, 2), kFaultConverter);
                if (!ok || *abort)
                    break;
                ptx::tc_fence_after();
                uint8_t *const row = p_tiles + c % l.p_buffers * l.p + i * kRowBytes;
                const int swizzle = (i & 7) << 4;
                const float2 mine = d.sum[i];
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
                            const float4 other = *reinterpret_cast<const float4 *>(&d.sum[at + j]);
                            const float one = (mine.x - other.x) + (mine.y - other.y);
                            const float two = (mine.x - other.z) + (mine.y - other.w);
                            f[e] = j <= i - at ? __uint_as_float(r[j]) * ex2(one) : 0.0f;
                            f[e + 1] = j + 1 <= i - at ? __uint_as_float(r[j + 1]) * ex2(two) : 0.0f;
                        }
                        store_parts<P::kMid>(row + (((at / 8 + u) << 4) ^ swizzle), kSlab, f);
                    }
                }
                ptx::fence_proxy_async_smem();
                ptx::tc_fence_before();
                ptx::mbar_arrive(&bar.p_full[b]);
            }
        }
    } else if (warp >= W::kOut && warp < W::kState) {
        // ---- inter and intra to y: lanes are values ----
        const int quarter = warp & 3, v = quarter * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        T *const first = p.out<T>(run.begin, head) + v0 + quarter * 32;
        T *const slice = reinterpret_cast<T *>(staging) + quarter * (C * 32);
        const int width = values - quarter * 32;  // of this warp's values
        for (int c = 0; outputs && c < chunks; ++c) {
            const int b = c & 1, ib = c % Col::kInters;
            const bool ok = wait(&bar.inter_full[ib], parity_of(c, Col::kInters), kFaultEpilogue) &&
                            wait(&bar.intra_full[b], parity_of(c, 2), kFaultEpilogue);
            if (!ok || *abort)
                break;
            ptx::tc_fence_after();
            const int len = min(run.end - run.begin - c * C, C);
            const Info &info = infos[c % kInfos];
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
                        const float4 since = *reinterpret_cast<const float4 *>(&info.since[e0 + e]);
                        const float some[4] = {since.x, since.y, since.z, since.w};
#pragma unroll
                        for (int n = 0; n < 4; ++n)
                            f[e + n] = p.scale * fmaf(__uint_as_float(past[e + n]), some[n],
                                                      __uint_as_float(r[e + n]));
                    }
                    if (!all_good) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            f[e] = e0 + e >= bad ? __uint_as_float(0x7fffffffu) : f[e];
                    }
                    if constexpr (sizeof(T) == 2) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            slice[(e0 + e) * 32 + lane] = Elem<T>::put(f[e]);
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
            ptx::mbar_arrive(&bar.y_free[b]);
            if constexpr (sizeof(T) == 2) {
                __syncwarp();
                if (aligned & 8) {
                    // 8 values of 8 rows at a time
                    const int col = (lane & 3) * 8;
#pragma unroll 2
                    for (int e = lane >> 2; e < len; e += 8) {
                        const Pack<T, 8> some = *reinterpret_cast<const Pack<T, 8> *>(slice + e * 32 + col);
                        if (col + 8 <= width)
                            store_pack<T, 8>(at + e * p.y_stride + col, some);
                    }
                } else if (lane < width) {
#pragma unroll 1
                    for (int e = 0; e < len; ++e)
                        at[e * p.y_stride + lane] = slice[e * 32 + lane];
                }
                __syncwarp();
            }
        }
    } else if (warp >= W::kState && warp < W::kLoad) {
        // ---- states: w v, S, and S as an operand ----
        const int quarter = warp & 3, k0 = ((warp - W::kState) >> 2) * 64;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const int v = quarter * 32 + lane, tid = threadIdx.x - W::kState * 32;
        const bool inside = v < values;
        float h[64];
        const int some = inside ? p.keys - k0 : 0;  // keys of this lane's h
        {
            const float *from = run.from + k0 * p.values + v;
            const int there = run.from ? some : 0;
#pragma unroll
            for (int n = 0; n < 64; ++n) {
                h[n] = n < there ? *from : 0.0f;
                from += p.values;
            }
        }
        float left = 0.0f;  // of the state, over chunk c
        // chunk c: its update joins the state; then w v of the next one, and the state for it
#pragma unroll 1
        for (int c = -1; c < chunks; ++c) {
            bool ok = true;
            if (c >= 0) {
                ok = wait(&bar.update_full, c & 1, kFaultConverter);
                if (!ok || *abort)
                    break;
                ptx::tc_fence_after();
#pragma unroll
                for (int n0 = 0; n0 < 64; n0 += 16) {
                    uint32_t r[16];
                    ptx::tmem_ld_32x32b_x16(tmem + lanes + Col::kUpdate + k0 + n0, r);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int n = 0; n < 16; ++n)
                        h[n0 + n] = fmaf(h[n0 + n], left, __uint_as_float(r[n]));
                }
                // (the next update may overwrite this one when w v is there)
                ptx::tc_fence_before();
            }
            const int next = c + 1;
            if (next == chunks)
                break;
            const int s = stage_of(next);
            const Decays &d = decays[s];
            if (!wait(&bar.full[s], turn_of(next), kFaultConverter))
                break;
            uint8_t *const tile = smem + s * l.stage + P::kIn * 2 * l.tile_k;
            left = d.all;
#pragma unroll 1
            for (int n0 = tid; n0 < l.tile_v / 16; n0 += 2 * W::kStates * 32) {
                float none = 0.0f;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int n = n0 + m * W::kStates * 32;
                    float f[8];
                    load_parts<P::kIn>(tile + n * 16, l.tile_v, f);
                    const float w = d.until[(n >> 3) & (C - 1)];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        none = fmaf(f[e], 0.0f, none);
                        f[e] *= w;
                    }
                    store_parts<kWeighted>(weighted + n * 16, l.tile_v, f);
                }
                if (none != 0.0f) {
#pragma unroll 1
                    for (int n = n0; n <= n0 + W::kStates * 32; n += W::kStates * 32) {
                        const int j = (n >> 3) & (C - 1);
                        not_finite<P::kIn>(tile + n * 16, l.tile_v,
                                           infos[next % kInfos].first_bad +
                                               n / (kSlab / 16) * 64 + ((n ^ j) & 7) * 8, j);
                    }
                }
            }
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(&bar.weighted_full[next % kWeights]);
            if (!outputs)
                continue;
            if (c >= 0) {
                // S of chunk c has been multiplied
                ok = wait(&bar.inter_full[c % Col::kInters], parity_of(c, Col::kInters),
                          kFaultConverter);
                if (!ok || *abort)
                    break;
                ptx::tc_fence_after();
            }
#pragma unroll
            for (int n0 = 0; n0 < 32; n0 += 8) {
                uint32_t r[P::kMid][8];
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    uint32_t parts[P::kMid];
                    split_pair_parts<P::kMid>(h[2 * (n0 + n)], h[2 * (n0 + n) + 1], parts);
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
            ptx::mbar_arrive(&bar.state_full);
        }
        if (run.to && !*abort) {
            float *to = run.to + k0 * p.values + v;
#pragma unroll
            for (int n = 0; n < 64; ++n) {
                if (n < some)
                    *to = h[n];
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
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                const int s = stage_of(c), b = c & 1;
                // a buffer of scores is free, and so is one of two of inter, when y of the
                // chunk before in it has been read
                if (!wait(&bar.full[s], turn_of(c), kFaultMma) ||
                    (c >= 2 && !wait(&bar.y_free[b], parity_of(c - 2, 2), kFaultMma)))
                    break;
                ptx::tc_fence_after();
                const uint64_t q_desc = ptx::sw128_desc(ptx::smem_u32(smem + s * l.stage));
                const uint64_t k_desc = q_desc + P::kIn * part_k;
                const uint64_t v_desc = ptx::sw128_desc(
                    ptx::smem_u32(smem + s * l.stage + P::kIn * 2 * l.tile_k), kSlab);
                const uint32_t scores = tmem + Col::kScores + C * b;
                multiply<P::kIn, P::kIn>(
                    leader, steps, [&](int i, int k) { return along_keys(q_desc, i, k); },
                    [&](int j, int k) { return along_keys(k_desc, j, k); },
                    [&](uint64_t a, uint64_t b_desc, bool more) {
                        ptx::mma_f16(scores, a, b_desc, idesc, more);
                    });
                if (leader)
                    ptx::mma_commit(&bar.scores_full[b]);
                if (!wait(&bar.state_full, c & 1, kFaultMma) ||
                    (Col::kInters == 1 && c > 0 &&
                     !wait(&bar.y_free[b ^ 1], parity_of(c - 1, 2), kFaultMma)))
                    break;
                ptx::tc_fence_after();
                const uint32_t inter = tmem + Col::kInter + C * (c % Col::kInters);
                multiply<P::kMid, P::kIn>(
                    leader, steps,
                    [&](int i, int k) { return tmem + Col::kState + i * (KP / 2) + k * 8; },
                    [&](int j, int k) { return along_keys(q_desc, j, k); },
                    [&](uint32_t a, uint64_t b_desc, bool more) {
                        ptx::mma_f16_tmem_a(inter, a, b_desc, idesc, more);
                    });
                if (leader)
                    ptx::mma_commit(&bar.inter_full[c % Col::kInters]);
                // (w v is there: values that are not finite have left V's tile)
                if (!wait(&bar.p_full[b], parity_of(c, 2), kFaultMma) ||
                    !wait(&bar.weighted_full[c % kWeights], parity_of(c, kWeights), kFaultMma))
                    break;
                ptx::tc_fence_after();
                const uint64_t p_desc = p_descs + c % l.p_buffers * (l.p >> 4);
                multiply<P::kIn, P::kMid>(
                    leader, C / 16, [&](int i, int k) { return v_desc + i * part_v + k * (2048 >> 4); },
                    [&](int j, int k) { return p_desc + j * (kSlab >> 4) + k * 2; },
                    [&](uint64_t a, uint64_t b_desc, bool more) {
                        ptx::mma_f16(scores, a, b_desc, idesc_v, more);
                    });
                if (leader) {
                    ptx::mma_commit(&bar.intra_full[b]);
                    ptx::mma_commit(&bar.empty[s]);
                }
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
            const uint64_t w_desc = ptx::sw128_desc(ptx::smem_u32(weighted), kSlab);
            for (int c = 0; c < chunks; ++c) {
                const int s = stage_of(c);
                if (!wait(&bar.full[s], turn_of(c), kFaultMma) ||
                    !wait(&bar.weighted_full[c % kWeights], parity_of(c, kWeights), kFaultMma))
                    break;
                ptx::tc_fence_after();
                const uint64_t k_desc = ptx::sw128_desc(
                    ptx::smem_u32(smem + s * l.stage) + P::kIn * l.tile_k, kSlab);
                multiply<kWeighted, P::kIn>(
                    leader, C / 16, [&](int i, int k) { return w_desc + i * (l.tile_v >> 4) + k * (2048 >> 4); },
                    [&](int j, int k) { return k_desc + j * (l.tile_k >> 4) + k * (2048 >> 4); },
                    [&](uint64_t a, uint64_t b_desc, bool more) {
                        ptx::mma_f16(tmem + Col::kUpdate, a, b_desc, idesc, more);
                    });
                if (leader) {
                    ptx::mma_commit(&bar.update_full);
                    ptx::mma_commit(&bar.empty[s]);
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
        double total = 0.0;
        for (int c = 0; c < chunks; ++c) {
            const int s = stage_of(c);
            const float n0 = decay_at(c + 1, 2 * lane), n1 = decay_at(c + 1, 2 * lane + 1);
            const bool ok = c < l.stages || wait(&bar.empty[s], turn_of(c) ^ 1, kFaultProducer);
            if (!ok)
                break;
            total += sum_decays(decays[s], infos[c % kInfos], g0, g1, lane);
            ptx::mbar_arrive(&bar.full[s]);
            g0 = n0;
            g1 = n1;
        }
        if (!outputs && lane == 0 && blockIdx.z == 0)
            *spans.left_of(p, blockIdx.x, head) = exp2f(static_cast<float>(total));
    } else if (warp >= W::kLoad && !test.withhold) {  // (failure test: nothing is loaded, so the waits for it run out)
        // ---- loaders ----
        const int tid = threadIdx.x - W::kLoad * 32;
        const auto arrive = [&](int c) {
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(&bar.full[stage_of(c)]);
        };
        int waiting = -1;  // the chunk whose copies have been asked for and not waited for
        for (int c = 0; c < chunks; ++c) {
            const int s = stage_of(c);
            if (c >= l.stages &&
                !__all_sync(0xffffffffu, ptx::mbar_try_wait(&bar.empty[s], turn_of(c) ^ 1))) {
                // nothing more can be asked for yet
                if (waiting >= 0) {
                    ptx::cp_async_wait_all();
                    arrive(waiting);
                    waiting = -1;
                }
                if (!wait(&bar.empty[s], turn_of(c) ^ 1, kFaultProducer))
                    break;
            }
            uint8_t *const at = smem + s * l.stage;
            const long long t0 = run.begin + static_cast<long long>(c) * C;
            const int len = min(run.end - run.begin - c * C, C);
#pragma unroll 1
            for (int which = outputs ? 0 : 1; which < 3; ++which) {
                const HeadRows &m = which == 0 ? p.q : which == 1 ? p.k : p.v;
                const bool of_v = which == 2;
                load_tile<T>(at + which * P::kIn * l.tile_k, of_v ? l.tile_v : l.tile_k,
                             m.row<T>(t0, head) + (of_v ? v0 : 0), m.stride,
                             aligned >> which & 1, len, of_v ? values : p.keys,
                             of_v ? l.slabs * 8 : KP / 8, tid);
            }
            ptx::cp_async_commit();
            if (waiting >= 0) {
                ptx::cp_async_wait<1>();
                arrive(waiting);
            }
            waiting = c;
        }
        ptx::cp_async_wait_all();
        if (waiting >= 0)
            arrive(waiting);
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == W::kOutIssue) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

template <typename T, int KP>
int launch(const AttentionArgs &p, const Spans &spans, bool outputs, cudaStream_t stream)
{
    using W = Warps<KP>;
    static SharedMemory memory;
    const Layout l = layout<T, KP>(p.values < 128 ? p.values : 128);
    int st = memory.allow(attention_kernel<T, KP>, 227 * 1024);
    if (st != LSTM_OK)
        return st;
    if (W::kShare) {
        // warpgroups that ask for more registers than the block has would wait for ever
        static const int registers = [] {
            cudaFuncAttributes a;
            return cudaFuncGetAttributes(&a, attention_kernel<T, KP>) == cudaSuccess ? a.numRegs : 0;
        }();
        if (registers != W::kRegisters)
            return fail(LSTM_E_CUDA, "lstm_linear_attention: %d registers a thread, built for %d",
                        registers, W::kRegisters);
    }
    unsigned *fault = fault_word();
    if (!fault)
        return fail(LSTM_E_CUDA, "cannot resolve the device fault word");
    if ((st = check_launch_injection("lstm_linear_attention")))
        return st;
    const auto in_place = [](const HeadRows &m) {
        return rows_aligned(m.at, m.stride, sizeof(T)) && m.head_stride * sizeof(T) % 16 == 0;
    };
    const bool y_vectors = rows_aligned(p.y, p.y_stride, sizeof(T)) && p.values % 8 == 0;
    const int aligned = in_place(p.q) | in_place(p.k) << 1 | in_place(p.v) << 2 | y_vectors << 3;
    const dim3 grid(static_cast<unsigned>(spans.tokens ? spans.units : p.seq.count),
                    static_cast<unsigned>(p.heads), static_cast<unsigned>((p.values + 127) / 128));
    attention_kernel<T, KP><<<grid, W::kThreads, l.total, stream>>>(
        p, spans, outputs, l, aligned, fault, kernel_test(kTestAttention));
    return cuda_status(cudaGetLastError(), "lstm_linear_attention launch");
}

template <typename T, int KP>
int launch_all(const AttentionArgs &p, const Spans &spans, cudaStream_t stream)
{
    int st;
    if (spans.tokens && ((st = launch<T, KP>(p, spans, false, stream)) ||
                         (st = launch_attention_join(p, spans, stream))))
        return st;
    return launch<T, KP>(p, spans, true, stream);
}

template <typename T>
int launch_keys(const AttentionArgs &p, const Spans &spans, cudaStream_t stream)
{
    return p.keys <= 64 ? launch_all<T, 64>(p, spans, stream) : launch_all<T, 128>(p, spans, stream);
}

}  // namespace prompts
}  // namespace lstm
