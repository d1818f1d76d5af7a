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
//  * 8 output warps turn scores into P, and inter and intra into y;
//  * 4 or 8 state warps hold S in registers (fp32, a lane per value), write w v, add the
//    update and hand S on as bf16;
//  * two threads issue the products, those of the outputs and those of the states, so that
//    neither chain waits for the other.
// bf16 inputs are exact operands.  P and S are rounded to bf16 for their products (an
// output of bf16 is rounded as coarsely itself); w v goes as two parts of bf16, so that
// what joins the state keeps 16 bits.  fp16 goes as two parts of bf16 (exact), so do P and
// S (which in fp16 itself would overflow); fp32 as three parts (exact), and so do P, S
// and w v.  Of two factors' parts those products are made that the other roundings leave
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
    static constexpr int kIn = 1, kMid = 1, kWeighted = 2;
};
template <>
struct Parts<__half> {
    static constexpr int kIn = 2, kMid = 2, kWeighted = 2;
};
template <>
struct Parts<float> {
    static constexpr int kIn = 3, kMid = 3, kWeighted = 3;
};

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
    float since[C];  // e^(c_i)
    float all;       // e^(c_64)
    float pad[3];
};

struct Layout {
    int slabs;         // of v: 64 values each
    int stages;
    int tile_k, tile_v, stage, weighted, p;  // bytes
    size_t total;
};

struct Barriers {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t scores_full[2], scores_free[2];
    uint64_t p_full, p_free, inter_full, inter_free, intra_full, state_full, weighted_full, update_full;
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
    l.weighted = P::kWeighted * l.tile_v;
    l.p = P::kMid * kSlab;
    // (products of 128 lanes read past tiles of 64, into the tile behind them)
    const size_t rest = l.weighted + l.p + kMaxStages * sizeof(Decays) + sizeof(Barriers) + 1024;
    l.stages = kMaxStages;
    while (l.stages > 1 && l.stages * l.stage + rest > 227 * 1024)
        --l.stages;
    l.total = l.stages * l.stage + rest;
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
    for (int i = 0; i < 8; ++i)
        f[i] = 0.0f;
#pragma unroll
    for (int k = N - 1; k >= 0; --k) {
        const uint4 u = *reinterpret_cast<const uint4 *>(at + k * apart);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] += low_float(w[i]);
            f[2 * i + 1] += high_float(w[i]);
        }
    }
}

// ---- loading ------------------------------------------------------------------------------
// Rows t0 .. t0 + 63 of a head into a tile of UNITS 16-byte units a row; rows from
// `len` and numbers from `width` on are zeros.  A thread keeps its unit and goes down the
// rows, so that swizzle and width are worked out once.
template <typename T, int UNITS>
__device__ __forceinline__ void load_tile(uint8_t *tile, int apart, const HeadRows &m, bool aligned,
                                          long long t0, int head, int len, int width, int first,
                                          int tid)
{
    constexpr int kDown = kLoaders / UNITS;  // rows of a turn, a multiple of 8
    static_assert(kDown % 8 == 0, "the swizzle of a thread's rows");
    const int u = tid % UNITS, r0 = tid / UNITS;
    const T *src = m.row<T>(t0 + r0, head) + first + u * 8;
    const long long down = kDown * m.stride;
    uint8_t *dst = tile + (u >> 3) * kSlab + r0 * kRowBytes + (((u & 7) ^ (r0 & 7)) << 4);
    const int there = min(max(width - u * 8, 0), 8);
    if constexpr (Parts<T>::kIn == 1) {
        if (aligned) {
            const uint32_t to = ptx::smem_u32(dst);
            const T *const some = m.row<T>(t0, head);  // an address where there is nothing to read
#pragma unroll
            for (int k = 0; k < C / kDown; ++k) {
                const bool in = r0 + k * kDown < len && there > 0;
                ptx::cp_async_16(to + k * kDown * kRowBytes, in ? src : some, in ? there * 2 : 0);
                src += down;
            }
            return;
        }
    }
    constexpr int kTogether = 4;  // rows in flight
#pragma unroll 1
    for (int k0 = 0; k0 < C / kDown; k0 += kTogether) {
        float f[kTogether][8];
#pragma unroll
        for (int k = 0; k < kTogether; ++k) {
            const bool in = k0 + k < C / kDown && r0 + (k0 + k) * kDown < len;
            if (aligned && there == 8) {
                constexpr int V = Elem<T>::kVector;
#pragma unroll
                for (int j = 0; j < 8; j += V) {
                    Pack<T, V> v = {};
                    if (in)
                        v = load_pack<T, V>(src + k * down + j);
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        f[k][j + e] = Elem<T>::get(v.v[e]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    f[k][j] = in && j < there ? Elem<T>::get(src[k * down + j]) : 0.0f;
            }
        }
#pragma unroll
        for (int k = 0; k < kTogether; ++k)
            if (k0 + k < C / kDown)
                store_parts<Parts<T>::kIn>(dst + (k0 + k) * kDown * kRowBytes, apart, f[k]);
        src += kTogether * down;
    }
}

// The sums of a chunk's log decays, two tokens a lane.
__device__ __forceinline__ void sum_decays(Decays &d, float g0, float g1, int lane)
{
    const auto log2_of = [](float g) {
        const double v = static_cast<double>(g) * 1.4426950408889634;
        return v < kLeast ? static_cast<double>(kLeast) : v;  // (a NaN stays)
    };
    const double a = log2_of(g0), b = log2_of(g1);
    double sum = a + b;
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
        const double other = __shfl_up_sync(0xffffffffu, sum, m);
        if (lane >= m)
            sum += other;
    }
    const double end = __shfl_sync(0xffffffffu, sum, 31);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const double c = k ? sum : sum - b;
        const int i = 2 * lane + k;
        const float hi = static_cast<float>(c);
        d.sum[i] = make_float2(hi, static_cast<float>(c - hi));
        d.until[i] = exp2f(static_cast<float>(end - c));
        d.since[i] = exp2f(hi) * (1.0f + 0.6931472f * static_cast<float>(c - hi));
    }
    if (lane == 0)
        d.all = exp2f(static_cast<float>(end));
}

// Value v's sum over the keys up to query t, from the tiles.
template <typename T>
__device__ __forceinline__ float seen_by(int t, int v, const uint8_t *p_tile, const uint8_t *v_tile,
                                      int tile_v)
{
    const auto number = [](const uint8_t *at) {
        return __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(at));
    };
    float sum = 0.0f;
#pragma unroll 1
    for (int j = 0; j <= t; ++j) {
        float pv = 0.0f, vv = 0.0f;
#pragma unroll
        for (int k = 0; k < Parts<T>::kMid; ++k)
            pv += number(p_tile + k * kSlab + t * kRowBytes + (((j >> 3) ^ (t & 7)) << 4) + (j & 7) * 2);
#pragma unroll
        for (int k = 0; k < Parts<T>::kIn; ++k)
            vv += number(v_tile + k * tile_v + (v >> 6) * kSlab + j * kRowBytes +
                         ((((v >> 3) & 7) ^ (j & 7)) << 4) + (v & 7) * 2);
        sum = fmaf(pv, vv, sum);
    }
    return sum;
}

// ---- the kernel ------------------------------------------------------------------------------
// Thread layout: output warps, state warps, two issuing warps, the decays' warp, loaders.
template <int KP>
struct Warps {
    static constexpr int kOut = 8;
    static constexpr int kState = 4 * (KP / 64);
    static constexpr int kIssue = kOut + kState;
    static constexpr int kDecay = kIssue + 2;
    static constexpr int kLoad = kDecay + 1;
    static constexpr int kThreads = (kLoad + 4 + 1) * 32;  // (whole warpgroups)
    // Registers: as the block is launched (65536 over its threads), and, with 128 keys, as
    // its warpgroups then share those of the launch, 768 x 80 = 256 x (72 + 104 + 64)
    static constexpr int kRegisters = KP > 64 ? 80 : 96;
    static constexpr bool kShare = KP > 64;
    static constexpr int kOutRegisters = 72, kStateRegisters = 104, kRestRegisters = 64;
    static_assert(kThreads % 128 == 0 && kIssue % 4 == 0, "warpgroups");
    static_assert(!kShare || kThreads * kRegisters == kOut * 32 * kOutRegisters +
                                                          kState * 32 * kStateRegisters +
                                                          (kThreads - kIssue * 32) * kRestRegisters,
                  "registers");
};
// Tensor memory: two buffers of scores (intra goes where its scores were), inter, the
// update, and S^T in up to three parts.
template <typename T, int KP>
struct Columns {
    static constexpr int kScores = 0, kInter = 128, kUpdate = 192, kState = 192 + KP;
    static constexpr int kUsed = kState + Parts<T>::kMid * KP / 2;
    static constexpr int kAlloc = kUsed <= 256 ? 256 : 512;
    static_assert(kUsed <= 512, "tensor memory");
};

// D = the products of parts that matter, over `steps` of the MOST blocks of 16 along the
// sum; a, b: an operand's descriptor for a part and a block, known but for a constant.
template <int MOST, int NA, int NB, typename A, typename B, typename M>
__device__ __forceinline__ void multiply(int steps, const A &a, const B &b, const M &mma)
{
    constexpr int most = NA > NB ? NA : NB;
    bool started = false;
    // the small products first
#pragma unroll
    for (int order = most - 1; order >= 0; --order)
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int j = order - i;
            if (j < 0 || j >= NB)
                continue;
#pragma unroll
            for (int k = 0; k < MOST; ++k)
                if (k < steps) {
                    mma(a(i, k), b(j, k), started || k > 0);
                }
            started = true;
        }
}

template <typename T, int KP>
__global__ void __launch_bounds__(Warps<KP>::kThreads, 1)
attention_kernel(const AttentionArgs p, const Layout l, const int aligned, unsigned *fault,
                 const KernelTest test)
{
    using W = Warps<KP>;
    using Col = Columns<T, KP>;
    using P = Parts<T>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *const weighted = smem + l.stages * l.stage;
    uint8_t *const p_tile = weighted + l.weighted;
    Decays *const decays = reinterpret_cast<Decays *>(p_tile + l.p);
    Barriers &bar = *reinterpret_cast<Barriers *>(decays + kMaxStages);
    volatile int *const abort = &bar.abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int head = blockIdx.y, v0 = blockIdx.z * 128;
    const int values = min(p.values - v0, 128);
    const int sequence = blockIdx.x;
    const int slot = sequence_slot(p.slots, sequence);
    Run run;
    run.begin = sequence_begin(p.seq, sequence);
    run.end = sequence_end(p.seq, sequence);
    run.to = slot >= 0 ? p.state_of(slot, head) + v0 : nullptr;
    run.from = run.to && sequence_resumes(p.slots, sequence) ? run.to : nullptr;
    const int chunks = (run.end - run.begin + C - 1) / C;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            ptx::mbar_init(&bar.full[s], kLoaders + 32);
            ptx::mbar_init(&bar.empty[s], 2 + W::kOut);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(&bar.scores_full[b], 1);
            ptx::mbar_init(&bar.scores_free[b], W::kOut * 32);
            ptx::mbar_init(&bar.done[b], 1);
        }
        ptx::mbar_init(&bar.p_full, W::kOut * 32);
        ptx::mbar_init(&bar.p_free, W::kOut);
        ptx::mbar_init(&bar.inter_full, 1);
        ptx::mbar_init(&bar.inter_free, W::kOut * 32);
        ptx::mbar_init(&bar.intra_full, 1);
        ptx::mbar_init(&bar.state_full, W::kState * 32);
        ptx::mbar_init(&bar.weighted_full, W::kState * 32);
        ptx::mbar_init(&bar.update_full, 1);
        bar.abort = 0;
        ptx::fence_mbar_init();
    }
    if (warp == W::kIssue) {
        ptx::tmem_alloc(&bar.tmem, Col::kAlloc);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = bar.tmem;
    const auto stage_of = [&](int c) { return c % l.stages; };
    const auto turn_of = [&](int c) { return static_cast<uint32_t>(c / l.stages) & 1; };
    const auto wait = [&](uint64_t *b, uint32_t parity, unsigned code) {
        return ptx::mbar_wait_bounded(b, parity, abort, fault, code, test.wait_limit_ns);
    };

    if constexpr (W::kShare) {
        if (warp < W::kOut)
            ptx::fewer_registers<W::kOutRegisters>();
        else if (warp < W::kIssue)
            ptx::more_registers<W::kStateRegisters>();
        else
            ptx::fewer_registers<W::kRestRegisters>();
    }
    if (warp < W::kOut) {
        // ---- outputs: scores to P, inter and intra to y ----
        // lanes are values, and queries of the scores; a warp takes half of the columns
        const int quarter = warp & 3, half = warp >> 2;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const int v = quarter * 32 + lane, i = v;
        T *y = p.out<T>(run.begin + half * 32, head) + v0 + v;
        for (int c = 0; c < chunks; ++c) {
            const int s = stage_of(c), b = c & 1;
            const uint32_t columns = tmem + lanes + Col::kScores + 64 * b + 32 * half;
            const Decays &d = decays[s];
            // (p_free: the warps that read P of the chunk before are done with it)
            bool ok = (c == 0 || wait(&bar.p_free, (c - 1) & 1, kFaultConverter)) &&
                      wait(&bar.full[s], turn_of(c), kFaultConverter) &&
                      wait(&bar.scores_full[b], (c >> 1) & 1, kFaultConverter);
            ok = __all_sync(0xffffffffu, ok) && !*abort;
            if (ok && quarter < 2) {
                ptx::tc_fence_after();
                uint8_t *const row = p_tile + i * kRowBytes;
                const int swizzle = (i & 7) << 4;
                if (half > quarter) {  // all keys of these columns come after all queries
                    const float none[8] = {};
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        store_parts<P::kMid>(row + (((half * 4 + u) << 4) ^ swizzle), kSlab, none);
                } else {
                    const float2 mine = d.sum[i];
                    uint32_t r[16];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        if (u % 2 == 0) {
                            ptx::tmem_ld_32x32b_x16(columns + u * 8, r);
                            ptx::tmem_ld_wait();
                        }
                        float f[8];
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            const int j = half * 32 + u * 8 + e;
                            const float4 other = *reinterpret_cast<const float4 *>(&d.sum[j]);
                            const float one = (mine.x - other.x) + (mine.y - other.y);
                            const float two = (mine.x - other.z) + (mine.y - other.w);
                            f[e] = j <= i ? __uint_as_float(r[u % 2 * 8 + e]) * ex2(one) : 0.0f;
                            f[e + 1] = j + 1 <= i ? __uint_as_float(r[u % 2 * 8 + e + 1]) * ex2(two) : 0.0f;
                        }
                        store_parts<P::kMid>(row + (((half * 4 + u) << 4) ^ swizzle), kSlab, f);
                    }
                }
                ptx::fence_proxy_async_smem();
                ptx::tc_fence_before();
            }
            ptx::mbar_arrive(&bar.p_full);
            ok = ok && wait(&bar.inter_full, c & 1, kFaultEpilogue) &&
                 wait(&bar.intra_full, c & 1, kFaultEpilogue);
            if (!__all_sync(0xffffffffu, ok) || *abort)
                break;
            ptx::tc_fence_after();
            const int len = run.end - run.begin - c * C - half * 32;
            const uint32_t inter = tmem + lanes + Col::kInter + 32 * half;
            uint32_t r[16];
            bool finite = true;
#pragma unroll
            for (int e0 = 0; e0 < 32; e0 += 16) {
                ptx::tmem_ld_32x32b_x16(columns + e0, r);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    finite = finite && fabsf(__uint_as_float(r[e])) <= 3.402823466e38f;
            }
            if (!__all_sync(0xffffffffu, finite || v >= values)) {
                // a value that is not finite met the zeros of P at the tokens before it: what
                // such a token may see is summed again
                const uint8_t *const tile = smem + s * l.stage + P::kIn * 2 * l.tile_k;
#pragma unroll 1
                for (int e = 0; e < 32; ++e) {
                    float sum = __uint_as_float(ptx::tmem_ld_32x32b_x1(columns + e));
                    const float past = __uint_as_float(ptx::tmem_ld_32x32b_x1(inter + e));
                    ptx::tmem_ld_wait();
                    if (v < values && e < len) {
                        if (!(fabsf(sum) <= 3.402823466e38f))
                            sum = seen_by<T>(half * 32 + e, v, p_tile, tile, l.tile_v);
                        y[e * p.y_stride] =
                            Elem<T>::put(p.scale * fmaf(past, d.since[half * 32 + e], sum));
                    }
                    __syncwarp();
                }
            } else {
                T *at = y;
#pragma unroll
                for (int e0 = 0; e0 < 32; e0 += 16) {
                    uint32_t past[16];
                    ptx::tmem_ld_32x32b_x16(columns + e0, r);
                    ptx::tmem_ld_32x32b_x16(inter + e0, past);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        if (v < values && e0 + e < len)
                            *at = Elem<T>::put(p.scale * fmaf(__uint_as_float(past[e]),
                                                              d.since[half * 32 + e0 + e],
                                                              __uint_as_float(r[e])));
                        at += p.y_stride;
                    }
                }
            }
            ptx::tc_fence_before();
            ptx::mbar_arrive(&bar.scores_free[b]);
            ptx::mbar_arrive(&bar.inter_free);
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(&bar.p_free);
                ptx::mbar_arrive(&bar.empty[s]);
            }
            y += C * p.y_stride;
        }
    } else if (warp < W::kIssue) {
        // ---- states: w v, S, and S as an operand ----
        const int quarter = warp & 3, k0 = ((warp - W::kOut) >> 2) * 64;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const int v = quarter * 32 + lane, tid = threadIdx.x - W::kOut * 32;
        const bool inside = v < values;
        float h[64];
#pragma unroll
        for (int n = 0; n < 64; ++n)
            h[n] = inside && run.from && k0 + n < p.keys
                       ? run.from[static_cast<long long>(k0 + n) * p.values + v]
                       : 0.0f;
        const auto hand_on = [&] {
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
        };
        if (chunks > 0)
            hand_on();
        for (int c = 0; c < chunks; ++c) {
            const int s = stage_of(c);
            const Decays &d = decays[s];
            bool ok = wait(&bar.full[s], turn_of(c), kFaultConverter);
            if (!__all_sync(0xffffffffu, ok))
                break;
            const uint8_t *const tile = smem + s * l.stage + P::kIn * 2 * l.tile_k;
            for (int n = tid; n < l.tile_v / 16; n += W::kState * 32) {
                float f[8];
                load_parts<P::kIn>(tile + n * 16, l.tile_v, f);
                const float w = d.until[(n >> 3) & (C - 1)];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[e] *= w;
                store_parts<P::kWeighted>(weighted + n * 16, l.tile_v, f);
            }
            const float all = d.all;
            ptx::fence_proxy_async_smem();
            ptx::tc_fence_before();
            ptx::mbar_arrive(&bar.weighted_full);
            ok = wait(&bar.update_full, c & 1, kFaultConverter);
            if (!__all_sync(0xffffffffu, ok) || *abort)
                break;
            ptx::tc_fence_after();
#pragma unroll
            for (int n0 = 0; n0 < 64; n0 += 16) {
                uint32_t r[16];
                ptx::tmem_ld_32x32b_x16(tmem + lanes + Col::kUpdate + k0 + n0, r);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int n = 0; n < 16; ++n)
                    h[n0 + n] = fmaf(h[n0 + n], all, __uint_as_float(r[n]));
            }
            if (c + 1 < chunks) {
                // S of the chunk before has been multiplied
                ok = wait(&bar.inter_full, c & 1, kFaultConverter);
                if (!__all_sync(0xffffffffu, ok) || *abort)
                    break;
                ptx::tc_fence_after();
                hand_on();
            }
        }
        if (run.to && inside && !*abort) {
#pragma unroll
            for (int n = 0; n < 64; ++n)
                if (k0 + n < p.keys)
                    run.to[static_cast<long long>(k0 + n) * p.values + v] = h[n];
        }
    } else if (warp == W::kIssue) {
        // ---- the outputs' products ----
        if (lane == 0) {
            constexpr uint32_t idesc = ptx::f16_idesc(128, C, true);
            constexpr uint32_t idesc_v = ptx::f16_idesc(128, C, true, true, false);
            const int steps = (p.keys + 15) / 16;
            // descriptors count 16 bytes: a part or a block further is a number added
            const uint64_t p_desc = ptx::sw128_desc(ptx::smem_u32(p_tile));
            const int part_k = l.tile_k >> 4, part_v = l.tile_v >> 4;
            const auto along_keys = [&](uint64_t desc, int part, int k) {
                return desc + part * part_k + (k >> 2) * (kSlab >> 4) + (k & 3) * 2;
            };
            const auto make_scores = [&](int c) {
                const int s = stage_of(c), b = c & 1;
                if (!wait(&bar.full[s], turn_of(c), kFaultMma) ||
                    (c >= 2 && !wait(&bar.scores_free[b], ((c >> 1) - 1) & 1, kFaultMma)))
                    return false;
                ptx::tc_fence_after();
                const uint64_t q_desc = ptx::sw128_desc(ptx::smem_u32(smem + s * l.stage));
                const uint64_t k_desc = q_desc + P::kIn * part_k;
                const uint32_t to = tmem + Col::kScores + 64 * b;
                multiply<KP / 16, P::kIn, P::kIn>(
                    steps, [&](int i, int k) { return along_keys(q_desc, i, k); },
                    [&](int j, int k) { return along_keys(k_desc, j, k); },
                    [&](uint64_t a, uint64_t b_desc, bool more) {
                        ptx::mma_f16(to, a, b_desc, idesc, more);
                    });
                ptx::mma_commit(&bar.scores_full[b]);
                return true;
            };
            // with one stage the next chunk's tiles come when this one's are done with
            const bool ahead = l.stages > 1;
            bool ok = chunks == 0 || make_scores(0);
            for (int c = 0; c < chunks && ok; ++c) {
                const int s = stage_of(c);
                const uint32_t q_at = ptx::smem_u32(smem + s * l.stage);
                const uint64_t q_desc = ptx::sw128_desc(q_at);
                const uint64_t v_desc = ptx::sw128_desc(q_at + P::kIn * 2 * l.tile_k, kSlab);
                if (!wait(&bar.state_full, c & 1, kFaultMma) ||
                    (c > 0 && !wait(&bar.inter_free, (c - 1) & 1, kFaultMma)))
                    break;
                ptx::tc_fence_after();
                multiply<KP / 16, P::kMid, P::kIn>(
                    steps,
                    [&](int i, int k) { return tmem + Col::kState + i * (KP / 2) + k * 8; },
                    [&](int j, int k) { return along_keys(q_desc, j, k); },
                    [&](uint32_t a, uint64_t b_desc, bool more) {
                        ptx::mma_f16_tmem_a(tmem + Col::kInter, a, b_desc, idesc, more);
                    });
                ptx::mma_commit(&bar.inter_full);
                if (ahead && c + 1 < chunks && !(ok = make_scores(c + 1)))
                    break;
                if (!wait(&bar.p_full, c & 1, kFaultMma))
                    break;
                ptx::tc_fence_after();
                multiply<C / 16, P::kIn, P::kMid>(
                    C / 16, [&](int i, int k) { return v_desc + i * part_v + k * (2048 >> 4); },
                    [&](int j, int k) { return p_desc + j * (kSlab >> 4) + k * 2; },
                    [&](uint64_t a, uint64_t b_desc, bool more) {
                        ptx::mma_f16(tmem + Col::kScores + 64 * (c & 1), a, b_desc, idesc_v, more);
                    });
                ptx::mma_commit(&bar.intra_full);
                ptx::mma_commit(&bar.empty[s]);
                if (!ahead && c + 1 < chunks)
                    ok = make_scores(c + 1);
            }
            // every product has completed before tensor memory is freed
            ptx::mma_commit(&bar.done[0]);
            ptx::mbar_wait_drain(&bar.done[0], 0, fault, kDefaultWaitLimitNs);
        }
    } else if (warp == W::kIssue + 1) {
        // ---- the states' products ----
        if (lane == 0) {
            constexpr uint32_t idesc = ptx::f16_idesc(128, KP, true, true, true);
            const uint64_t w_desc = ptx::sw128_desc(ptx::smem_u32(weighted), kSlab);
            for (int c = 0; c < chunks; ++c) {
                const int s = stage_of(c);
                if (!wait(&bar.full[s], turn_of(c), kFaultMma) ||
                    !wait(&bar.weighted_full, c & 1, kFaultMma))
                    break;
                ptx::tc_fence_after();
                const uint64_t k_desc = ptx::sw128_desc(
                    ptx::smem_u32(smem + s * l.stage) + P::kIn * l.tile_k, kSlab);
                multiply<C / 16, P::kWeighted, P::kIn>(
                    C / 16, [&](int i, int k) { return w_desc + i * (l.tile_v >> 4) + k * (2048 >> 4); },
                    [&](int j, int k) { return k_desc + j * (l.tile_k >> 4) + k * (2048 >> 4); },
                    [&](uint64_t a, uint64_t b_desc, bool more) {
                        ptx::mma_f16(tmem + Col::kUpdate, a, b_desc, idesc, more);
                    });
                ptx::mma_commit(&bar.update_full);
                ptx::mma_commit(&bar.empty[s]);
            }
            ptx::mma_commit(&bar.done[1]);
            ptx::mbar_wait_drain(&bar.done[1], 0, fault, kDefaultWaitLimitNs);
        }
    } else if (warp == W::kDecay) {
        const auto decay_at = [&](int c, int i) {
            const int t = run.begin + c * C + i;
            return t < run.end ? __ldg(p.decay + t * p.decay_stride + head) : 0.0f;
        };
        float g0 = decay_at(0, 2 * lane), g1 = decay_at(0, 2 * lane + 1);
        for (int c = 0; c < chunks; ++c) {
            const int s = stage_of(c);
            const float n0 = decay_at(c + 1, 2 * lane), n1 = decay_at(c + 1, 2 * lane + 1);
            const bool ok = c < l.stages || wait(&bar.empty[s], turn_of(c) ^ 1, kFaultProducer);
            if (!__all_sync(0xffffffffu, ok))
                break;
            sum_decays(decays[s], g0, g1, lane);
            ptx::mbar_arrive(&bar.full[s]);
            g0 = n0;
            g1 = n1;
        }
    } else if (warp < W::kLoad + 4 && !test.withhold) {  // (failure test: nothing is loaded, so the waits for it run out)
        // ---- loaders ----
        const int tid = threadIdx.x - W::kLoad * 32;
        const auto arrive = [&](int c) {
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(&bar.full[stage_of(c)]);
        };
        int waiting = -1;  // the chunk whose copies have been asked for and not waited for
        for (int c = 0; c < chunks; ++c) {
            const int s = stage_of(c);
            if (c >= l.stages && !ptx::mbar_try_wait(&bar.empty[s], turn_of(c) ^ 1)) {
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
            load_tile<T, KP / 8>(at, l.tile_k, p.q, aligned & 1, t0, head, len, p.keys, 0, tid);
            load_tile<T, KP / 8>(at + P::kIn * l.tile_k, l.tile_k, p.k, aligned & 2, t0, head, len,
                                 p.keys, 0, tid);
            uint8_t *const v_at = at + P::kIn * 2 * l.tile_k;
            if (l.slabs == 1)
                load_tile<T, 8>(v_at, l.tile_v, p.v, aligned & 4, t0, head, len, values, v0, tid);
            else
                load_tile<T, 16>(v_at, l.tile_v, p.v, aligned & 4, t0, head, len, values, v0, tid);
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
    if (warp == W::kIssue) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, Col::kAlloc);
    }
}

template <typename T, int KP>
int launch(const AttentionArgs &p, cudaStream_t stream)
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
    const int aligned = in_place(p.q) | in_place(p.k) << 1 | in_place(p.v) << 2;
    const dim3 grid(static_cast<unsigned>(p.seq.count), static_cast<unsigned>(p.heads),
                    static_cast<unsigned>((p.values + 127) / 128));
    attention_kernel<T, KP><<<grid, W::kThreads, l.total, stream>>>(
        p, l, aligned, fault, kernel_test(kTestAttention));
    return cuda_status(cudaGetLastError(), "lstm_linear_attention launch");
}

template <typename T>
int launch_keys(const AttentionArgs &p, cudaStream_t stream)
{
    return p.keys <= 64 ? launch<T, 64>(p, stream) : launch<T, 128>(p, stream);
}

}  // namespace prompts
}  // namespace lstm
