// Dense product with bias, activation and residual in its epilogue:
//     y[r][n] = act(sum_k x[r][k] w[n][k] + bias[n]) + residual[r][n].
//
// One kernel (sm_103a) of warps with one task each:
//  * warp 0 (one thread) streams K blocks of 64 (128 bytes, 128-byte swizzle) of the
//    tile's two operands through a ring of stages with TMA;
//  * warp 1 (one thread) issues tcgen05.mma kind::f16, M = 128, into a tensor-memory
//    accumulator;
//  * warps 2-9 read a finished accumulator (a lane per row of the tile, half of the columns
//    each), add the bias, apply the activation, add the residual and store.
// Many rows: M are 128 rows of x and N up to 256 rows of w; one CTA an SM walks over
// the tiles, and a second accumulator lets a tile's epilogue run under the next tile's
// products.  An SM gets 64 bytes a cycle from L2, so a tile of 128 x 256 waits for its
// loads (48 KB a K block: 768 cycles, of which the products take 524): large products go to
// pairs of SMs (cta_group::2), which share a tile of 256 x 256 and load half of w's rows
// each.  2048 x 2048 x 8192 takes 54 us (59 by single SMs), 12288 x 4096 x 4096 275 us (294;
// at 1.5 PFLOP/s the card runs into its power limit).
// Few rows (at most kFewRows): the operands change places, M are 128 rows of w and N the 16
// to 64 rows of x, so that a tile's 128 lanes all work and w streams once (64 x 4096 x 16384:
// 29 us, 20 at the memory's rate).  Up to three rows go without tensor cores (dense_few.cu).
// Where a call has fewer tiles than SMs, the CTAs of a cluster take a part of K each, and
// each then joins its share of the tile's sums through distributed shared memory, in the
// order of the parts.
//
// fp32 goes as bf16: x = x1 + x2 + x3 exactly, each the nearest to what the ones before it
// leave, and of the nine products of two numbers' parts the six that reach 2^-24 of the
// product are summed, the small ones first.  The split, and a copy to
// 16-byte pitches of 16-bit operands that TMA cannot read in place, is a kernel before.
#include <math_constants.h>

#include "dense.cuh"

namespace lstm {
namespace {

constexpr int BM = 128;
constexpr int BK = 64;
constexpr int A_BYTES = BM * BK * 2;
constexpr int kFewRows = 64;
constexpr int kMaxStages = 12;
constexpr int kParts = 3;      // of an fp32 number
constexpr int kProducts = 6;   // of two of them
constexpr int EPILOGUE_WARPS = 8;
constexpr int THREADS = 64 + EPILOGUE_WARPS * 32;
constexpr int PRODUCER_WARP = 0, MMA_WARP = 1;
constexpr int SLICE_BYTES = 32 * 128;  // a warp's 32 rows of 128 bytes on their way out

struct DenseArgs {
    const void *x, *w;
    long long x_stride, w_stride;
    const float *bias;
    const void *residual;
    void *y;
    long long residual_stride, y_stride;
    int rows, in, out;
    int activation;
    int products;         // 1, or kProducts
    int split;            // CTAs of a cluster, each a part of K
    bool store_boxes;     // y takes TMA stores
    bool vectors;         // the residual's rows start on 16-byte boundaries
    bool whole;           // so does the bias
    int group;            // tiles down M that run side by side
};

// Which parts of x and w the p-th product takes.
__host__ __device__ constexpr int part_of_x(int p) { return p == 0 ? 2 : p == 1 || p == 3 ? 1 : 0; }
__host__ __device__ constexpr int part_of_w(int p) { return p == 2 ? 2 : p == 1 || p == 4 ? 1 : 0; }

template <int BN_, bool SWAP_, bool PAIR_ = false>
struct Shape {
    static constexpr int BN = BN_;
    static constexpr bool SWAP = SWAP_, PAIR = PAIR_;
    static constexpr int CTAS = PAIR ? 2 : 1;  // of a tile, 128 lanes of M each
    static constexpr int B_ROWS = BN / CTAS;
    static constexpr int B_BYTES = B_ROWS * BK * 2;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int DATA_BYTES = 224 * 1024;
    static constexpr int SLICES = PAIR ? 2 : 1;  // a warp's, in turn
    static constexpr int OUT_BYTES = SWAP ? 0 : EPILOGUE_WARPS * SLICES * SLICE_BYTES;
    static constexpr int FIT = (DATA_BYTES - OUT_BYTES) / STAGE_BYTES;
    static constexpr int STAGES = FIT < kMaxStages ? FIT : kMaxStages;
    static constexpr int RING_BYTES = STAGES * STAGE_BYTES;
    static constexpr int ACCS = SWAP ? 1 : 2;
    static constexpr int TMEM_COLS = ACCS * BN < 32 ? 32 : ACCS * BN;
    static constexpr int CW = BN < 32 ? BN : 32;  // columns read at a time
    static constexpr size_t SMEM_BYTES = RING_BYTES + OUT_BYTES + 256 + 1024;
    // a tile's sums on their way to the other CTAs of a cluster, rows of y one after another
    static constexpr int SUM_ROWS = SWAP ? BN : BM, SUM_COLS = SWAP ? BM : BN, SUM_PITCH = SUM_COLS + 4;
    static_assert(STAGES >= 4 && SUM_ROWS * SUM_PITCH * 4 <= RING_BYTES, "ring");
    static_assert(STAGE_BYTES % 1024 == 0, "stage alignment");
};

template <int N>
__device__ __forceinline__ void read_columns(uint32_t taddr, float (&f)[N])
{
    uint32_t r[N];
    if constexpr (N == 32)
        ptx::tmem_ld_32x32b_x32(taddr, r);
    else
        ptx::tmem_ld_32x32b_x16(taddr, r);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < N; ++i)
        f[i] = __uint_as_float(r[i]);
}

// fp32's own sum where that of the parts is infinite: parts have either sign, so that a product
// beyond 2^136 overflows to an infinity of either sign before its largest part joins the sum.
__device__ __forceinline__ float overflowed(const float *x, const float *w, int in)
{
    float sum = 0.0f;
#pragma unroll 4
    for (int k = 0; k < in; ++k)
        sum = fmaf(__ldg(x + k), __ldg(w + k), sum);
    return sum;
}
// The same for `count` columns of an accumulator, by all lanes of a warp: column c is the sum of
// rows x + c * dx and w + c * dw, and the lane has `there` of them.  Out of line and back through
// tensor memory, since this is for few results and takes no register of the others'; its callers
// read the columns once more in a loop (where the second reading had code of its own, the
// activations lost a third of their speed).
__device__ __noinline__ void mend_columns(uint32_t taddr, int count, int there, const float *x,
                                          const float *w, long long dx, long long dw, int in)
{
    for (int c = 0; c < count; ++c) {
        uint32_t v;
        ptx::tmem_ld_32x32b_x1(taddr + c, v);
        ptx::tmem_ld_wait();
        if (fabsf(__uint_as_float(v)) == CUDART_INF_F && c < there)
            v = __float_as_uint(overflowed(x + c * dx, w + c * dw, in));
        __syncwarp();
        ptx::tmem_st_32x32b_x1(taddr + c, v);
    }
    ptx::tmem_st_wait();
}
__device__ __forceinline__ bool infinite(float v) { return fabsf(v) == CUDART_INF_F; }
// of any lane of the warp
template <int N>
__device__ __forceinline__ bool any_infinite(const float (&f)[N])
{
    bool any = false;
#pragma unroll
    for (int j = 0; j < N; ++j)
        any |= infinite(f[j]);
    return __builtin_expect(__any_sync(0xffffffffu, any), 0);
}

template <class S, typename T>
__global__ void __launch_bounds__(THREADS, 1)
dense_kernel(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap b_map,
             const __grid_constant__ CUtensorMap y_map, const DenseArgs p, uint32_t idesc,
             long long tiles, int tiles_m, unsigned *fault, KernelTest test)
{
    constexpr int BN = S::BN, STAGES = S::STAGES, CW = S::CW;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *out_slices = smem + S::RING_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(out_slices + S::OUT_BYTES);
    uint64_t *empty = full + kMaxStages;
    uint64_t *acc_full = empty + kMaxStages;  // [2]
    uint64_t *acc_empty = acc_full + 2;       // [2]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_empty + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    // of a pair's first CTA: the K blocks that the second one has asked for, and that it asks for
    // no more
    volatile uint32_t *peer_total = tmem_slot + 2;
    uint64_t *peer_done = reinterpret_cast<uint64_t *>(tmem_slot + 4);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        ptx::mbar_init(peer_done, 1);
        for (int s = 0; s < STAGES; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(&acc_full[a], 1);
            ptx::mbar_init(&acc_empty[a], EPILOGUE_WARPS * S::CTAS);
        }
        *abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&a_map);
        ptx::prefetch_tensormap(&b_map);
    }
    if (warp == MMA_WARP) {
        if constexpr (S::PAIR) {
            ptx::tmem_alloc_pair(tmem_slot, S::TMEM_COLS);
            ptx::tmem_relinquish_pair();
        } else {
            ptx::tmem_alloc(tmem_slot, S::TMEM_COLS);
            ptx::tmem_relinquish();
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (S::PAIR) {
        // the peer's barriers are there before anything arrives on them
        ptx::cluster_arrive_release();
        ptx::cluster_wait_acquire();
    }
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    ptx::griddep_wait();  // (the copies of this call's operands)
    const uint32_t rank = S::PAIR ? ptx::cluster_ctarank() : 0;

    // this CTA's tiles, and its part of their K blocks
    const int part = !S::PAIR && p.split > 1 ? static_cast<int>(ptx::cluster_ctarank()) : 0;
    const int together = S::PAIR ? 2 : p.split;
    const long long first = blockIdx.x / together, step = gridDim.x / together;
    const int kblocks = (p.in + BK - 1) / BK, all = kblocks * p.products;
    const int kb_begin = static_cast<int>(static_cast<long long>(all) * part / p.split);
    const int kb_end = static_cast<int>(static_cast<long long>(all) * (part + 1) / p.split);
    const auto place = [&](long long t, int *m, int *n) {
        // groups of tiles down M, inside them down M first
        const long long tiles_n = tiles / tiles_m;
        const long long g = t / (p.group * tiles_n), in_group = t - g * p.group * tiles_n;
        const int tall = min(p.group, tiles_m - static_cast<int>(g) * p.group);
        *m = ((static_cast<int>(g) * p.group + static_cast<int>(in_group % tall)) * S::CTAS + rank) * BM;
        *n = static_cast<int>(in_group / tall) * BN;
    };
    // What a tile takes counts beside the limit: with a K of millions its products outlast any, and
    // so do fp32 sums that are made again.
    const uint64_t limit_ns =
        test.wait_limit_ns + static_cast<uint64_t>(kb_end - kb_begin) * (sizeof(T) == 4 ? 1000000 : 10000);
    int issued = 0;  // K blocks, as far as they matter at the end: the last STAGES
    uint32_t total = 0;
    int committed = 0;
    // the ring's next stage, and the parity of its turn (no divisions: a K block takes the
    // tensor core some 260 to 530 cycles, and one thread has to keep up)
    int s = 0;
    uint32_t turn = 0;
    const auto advance = [&] {
        if (++s == STAGES) {
            s = 0;
            turn ^= 1;
        }
    };

    if (warp == PRODUCER_WARP) {
        // failure test (`withhold`): nothing is loaded, so the waits for it run out
        if (lane == 0 && !test.withhold) {
            const int a_rows = S::SWAP ? p.out : p.rows, b_rows = S::SWAP ? p.rows : p.out;
            bool ok = true;
            for (long long t = first; t < tiles && ok && !*abort_flag; t += step) {
                int m0, n0;
                place(t, &m0, &n0);
                int product = kb_begin / kblocks, k = kb_begin - product * kblocks;
                for (int kb = kb_begin; kb < kb_end; ++kb) {
                    // (a stage's first use finds it free)
                    if (!ptx::mbar_wait_bounded(&empty[s], turn ^ 1, abort_flag, fault,
                                                kFaultProducer, limit_ns)) {
                        ok = false;
                        break;
                    }
                    int ax = m0, bx = n0 + rank * S::B_ROWS;
                    if (p.products > 1) {  // behind the rows of the parts before these
                        ax += (S::SWAP ? part_of_w(product) : part_of_x(product)) * a_rows;
                        bx += (S::SWAP ? part_of_x(product) : part_of_w(product)) * b_rows;
                    }
                    uint8_t *st = smem + s * S::STAGE_BYTES;
                    if constexpr (S::PAIR) {
                        // both CTAs' bytes count on the first one's barrier
                        const uint32_t bar = ptx::map_to_rank(ptx::smem_u32(&full[s]), 0);
                        if (rank == 0)
                            ptx::mbar_arrive_expect_tx(&full[s], 2 * S::STAGE_BYTES);
                        ptx::tma_load_2d_pair(st, &a_map, bar, k * BK, ax);
                        ptx::tma_load_2d_pair(st + A_BYTES, &b_map, bar, k * BK, bx);
                    } else {
                        ptx::mbar_arrive_expect_tx(&full[s], S::STAGE_BYTES);
                        ptx::tma_load_2d(st, &a_map, &full[s], k * BK, ax);
                        ptx::tma_load_2d(st + A_BYTES, &b_map, &full[s], k * BK, bx);
                    }
                    if (++k == kblocks) {
                        k = 0;
                        ++product;
                    }
                    if (issued < STAGES)
                        ++issued;
                    ++total;
                    advance();
                }
            }
        }
        if (S::PAIR && lane == 0 && rank > 0) {
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(
                             ptx::map_to_rank(ptx::smem_u32(const_cast<uint32_t *>(peer_total)), 0)),
                         "r"(total)
                         : "memory");
            ptx::mbar_arrive_cluster(ptx::map_to_rank(ptx::smem_u32(peer_done), 0));
        }
    } else if (warp == MMA_WARP && rank > 0) {
        // (the first CTA of a pair issues for both, and waits for both at the end)
    } else if (warp == MMA_WARP) {
        const bool leader = ptx::elect_one();
        const uint64_t a_desc = ptx::sw128_desc(ptx::smem_u32(smem));
        for (long long t = first; t < tiles && !*abort_flag; t += step) {
            const int a = committed % S::ACCS;
            const uint32_t use = static_cast<uint32_t>(committed / S::ACCS);
            bool ok = use == 0 || ptx::mbar_wait_bounded(&acc_empty[a], (use - 1) & 1, abort_flag, fault,
                                                         kFaultMma, limit_ns, S::PAIR);
            if (!__all_sync(0xffffffffu, ok))
                break;
            ptx::tc_fence_after();
            const uint32_t d = tmem + a * BN;
            for (int kb = kb_begin; kb < kb_end; ++kb) {
                ok = ptx::mbar_wait_bounded(&full[s], turn, abort_flag, fault, kFaultMma,
                                            limit_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                ptx::tc_fence_after();
                if (leader) {
                    const uint64_t at = a_desc + s * (S::STAGE_BYTES >> 4);
#pragma unroll
                    for (int j = 0; j < BK / 16; ++j)
                        ptx::mma_f16<S::CTAS>(d, at + 2 * j, at + (A_BYTES >> 4) + 2 * j, idesc,
                                              kb != kb_begin || j != 0);
                    ptx::mma_commit<S::CTAS>(&empty[s]);
                }
                advance();
            }
            if (leader)
                ptx::mma_commit<S::CTAS>(&acc_full[a]);  // also when stopping: frees the epilogue
            ++committed;
            if (!ok)
                break;
        }
    } else {
        // epilogue: this warp reads the tensor-memory lanes (rows of the tile) 32q..32q+31, of
        // every other slice of columns
        const int q = warp & 3, turn = (warp - 2) >> 2;
        constexpr int TURNS = EPILOGUE_WARPS / 4;
        const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
        uint8_t *const slices = out_slices + (warp - 2) * S::SLICES * SLICE_BYTES;
        int sent = 0;
        T *const y = static_cast<T *>(p.y);
        const T *const residual = static_cast<const T *>(p.residual);
        int count = 0;
        for (long long t = first; t < tiles; t += step, ++count) {
            int m0, n0;
            place(t, &m0, &n0);
            const int a = count % S::ACCS;
            const bool got = ptx::mbar_wait_bounded(&acc_full[a], (count / S::ACCS) & 1, abort_flag,
                                                    fault, kFaultEpilogue, limit_ns);
            // tcgen05.ld is warp-collective: continue only if every lane may
            const bool ok = __all_sync(0xffffffffu, got) && !*abort_flag;
            ptx::tc_fence_after();
            const uint32_t acc = tmem + lane_base + a * BN;
            if (p.split > 1) {
                // (every load of the ring has landed and been multiplied: the sums take its place)
                float *const sums = reinterpret_cast<float *>(smem);
                if (ok) {
#pragma unroll 1
                    for (int c = turn * CW; c < BN; c += TURNS * CW) {
                        float f[CW];
                        read_columns<CW>(acc + c, f);
                        if constexpr (S::SWAP) {
#pragma unroll
                            for (int j = 0; j < CW; ++j)
                                sums[(c + j) * S::SUM_PITCH + q * 32 + lane] = f[j];
                        } else {
#pragma unroll
                            for (int j = 0; j < CW; j += 4)
                                *reinterpret_cast<float4 *>(sums + (q * 32 + lane) * S::SUM_PITCH + c + j) =
                                    make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
                        }
                    }
                }
                ptx::cluster_arrive_release();
                ptx::cluster_wait_acquire();
                if (!ok)
                    break;
                // each CTA joins its share of the tile, four numbers of a row at a time, the
                // parts in their order
                constexpr int QUADS = S::SUM_COLS / 4, ALL = S::SUM_ROWS * QUADS;
                const int high = S::SWAP ? p.rows - n0 : p.rows - m0;
                const int wide = S::SWAP ? p.out - m0 : p.out - n0;
                const int row0 = S::SWAP ? n0 : m0, col0 = S::SWAP ? m0 : n0;
                const uint32_t base = ptx::smem_u32(sums);
                for (int u = part * (ALL / p.split) + static_cast<int>(threadIdx.x) - 64;
                     u < (part + 1) * (ALL / p.split); u += EPILOGUE_WARPS * 32) {
                    const int row = u / QUADS, col = u % QUADS * 4;
                    if (row >= high || col >= wide)
                        continue;
                    const uint32_t at = base + (row * S::SUM_PITCH + col) * 4;
                    float f[4] = {};
                    bool any = false;
#pragma unroll 4
                    for (int k = 0; k < p.split; ++k) {
                        float v[4];
                        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                                     : "r"(ptx::map_to_rank(at, k)));
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            f[j] += v[j];
                            any |= sizeof(T) == 4 && infinite(v[j]);
                        }
                    }
                    const long long r = row0 + row;
                    const int n = col0 + col, there = min(4, wide - col);
                    if (any) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j < there && !(fabsf(f[j]) < CUDART_INF_F))
                                f[j] = overflowed(static_cast<const float *>(p.x) + r * p.x_stride,
                                                  static_cast<const float *>(p.w) + (n + j) * p.w_stride,
                                                  p.in);
                    }
                    T *const to = y + r * p.y_stride + n;
                    const T *const res = residual ? residual + r * p.residual_stride + n : nullptr;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < there) {
                            const float bias = p.bias ? __ldg(p.bias + n + j) : 0.0f;
                            float v = activate<sizeof(T) == 4>(p.activation, f[j] + bias);
                            if (res)
                                v += Elem<T>::get(res[j]);
                            to[j] = Elem<T>::put(v);
                        }
                }
                ptx::tc_fence_before();
                continue;
            }
            if (!ok)
                break;
            if constexpr (S::SWAP) {
                // a lane's row of the tile is one column of y, its columns are rows of y
                const int n = m0 + q * 32 + lane;
                const float bias = p.bias && n < p.out ? __ldg(p.bias + n) : 0.0f;
                for (int c0 = turn * CW; c0 < BN && n0 + c0 < p.rows; c0 += TURNS * CW) {
                    float f[CW];
                    bool first = true;
#pragma unroll 1
                    while (true) {
                        read_columns<CW>(acc + c0, f);
                        if (!(sizeof(T) == 4 && first && any_infinite(f)))
                            break;
                        first = false;
                        const long long r = n0 + c0;
                        mend_columns(acc + c0, CW, n < p.out ? p.rows - n0 - c0 : 0,
                                     static_cast<const float *>(p.x) + r * p.x_stride,
                                     static_cast<const float *>(p.w) + n * p.w_stride, p.x_stride, 0,
                                     p.in);
                    }
#pragma unroll
                    for (int j = 0; j < CW; ++j) {
                        const long long r = n0 + c0 + j;
                        if (r < p.rows && n < p.out) {
                            float v = activate<sizeof(T) == 4>(p.activation, f[j] + bias);
                            if (residual)
                                v += Elem<T>::get(residual[r * p.residual_stride + n]);
                            y[r * p.y_stride + n] = Elem<T>::put(v);
                        }
                    }
                }
            } else {
                constexpr int V = Elem<T>::kVector;
                const int r0 = m0 + q * 32;
                const long long r = r0 + lane;
                // slices of 128 bytes of a row; 16-byte unit u of row r lies at u ^ (r % 8)
                constexpr int WIDE = 128 / static_cast<int>(sizeof(T));
                constexpr int TOGETHER = 16;  // numbers a lane has in flight, of WIDE
                uint8_t *buf = slices;
                const auto in_slice = [&](int row, int col) {
                    return reinterpret_cast<T *>(buf + row * 128 + (((col / V) ^ (row & 7)) << 4)) + col % V;
                };
                const int high = min(32, p.rows - r0);
                for (int c0 = turn * WIDE; c0 < BN && n0 + c0 < p.out; c0 += TURNS * WIDE) {
                    // the store that last used this buffer has read it
                    if (p.store_boxes) {
                        buf = slices + (sent++ & (S::SLICES - 1)) * SLICE_BYTES;
                        if (lane == 0)
                            ptx::bulk_wait_group_read<S::SLICES - 1>();
                        __syncwarp();
                    }
                    const int wide = min(WIDE, p.out - (n0 + c0));
                    if (residual && !p.vectors) {
                        // row by row, each as its neighbours in memory
                        const T *from = residual + r0 * p.residual_stride + n0 + c0;
#pragma unroll 1
                        for (int k0 = 0; k0 < WIDE; k0 += TOGETHER) {
                            T v[TOGETHER];
#pragma unroll
                            for (int k = 0; k < TOGETHER; ++k) {
                                const int row = (k0 + k) / (WIDE / 32), col = (k0 + k) % (WIDE / 32) * 32 + lane;
                                if (row < high && col < wide)
                                    v[k] = from[row * p.residual_stride + col];
                            }
#pragma unroll
                            for (int k = 0; k < TOGETHER; ++k)
                                *in_slice((k0 + k) / (WIDE / 32), (k0 + k) % (WIDE / 32) * 32 + lane) = v[k];
                        }
                        __syncwarp();
                    }
#pragma unroll
                    for (int h = 0; h < WIDE; h += CW) {
                        const int n = n0 + c0 + h;
                        float f[CW];
                        bool first = true;
#pragma unroll 1
                        while (true) {
                            read_columns<CW>(acc + c0 + h, f);
                            if (!(sizeof(T) == 4 && first && any_infinite(f)))
                                break;
                            first = false;
                            mend_columns(acc + c0 + h, CW, r < p.rows ? p.out - n : 0,
                                         static_cast<const float *>(p.x) + r * p.x_stride,
                                         static_cast<const float *>(p.w) + n * p.w_stride, 0,
                                         p.w_stride, p.in);
                        }
                        if (p.bias && p.whole && n + CW <= p.out) {
#pragma unroll
                            for (int j = 0; j < CW; j += 4) {
                                const float4 b = __ldg(reinterpret_cast<const float4 *>(p.bias + n + j));
                                f[j] += b.x;
                                f[j + 1] += b.y;
                                f[j + 2] += b.z;
                                f[j + 3] += b.w;
                            }
                        } else if (p.bias) {
#pragma unroll
                            for (int j = 0; j < CW; ++j)
                                f[j] += n + j < p.out ? __ldg(p.bias + n + j) : 0.0f;
                        }
                        if (p.activation != LSTM_ACT_NONE) {
#pragma unroll
                            for (int j = 0; j < CW; ++j)
                                f[j] = activate<sizeof(T) == 4>(p.activation, f[j]);
                        }
                        if (residual) {
                            const T *res = residual + r * p.residual_stride + n;
#pragma unroll
                            for (int j = 0; j < CW; j += V) {
                                Pack<T, V> v = {};
                                if (!p.vectors)
                                    v = *reinterpret_cast<const Pack<T, V> *>(in_slice(lane, h + j));
                                else if (r < p.rows && n + j < p.out)
                                    v = *reinterpret_cast<const Pack<T, V> *>(res + j);
#pragma unroll
                                for (int i = 0; i < V; ++i)
                                    f[j + i] += Elem<T>::get(v.v[i]);
                            }
                        }
#pragma unroll
                        for (int j = 0; j < CW; j += V) {
                            float some[V];
#pragma unroll
                            for (int i = 0; i < V; ++i)
                                some[i] = f[j + i];
                            *reinterpret_cast<Pack<T, V> *>(in_slice(lane, h + j)) = pack<T, V>(some);
                        }
                    }
                    if (p.store_boxes) {
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            if (r0 < p.rows)
                                ptx::tma_store_2d(&y_map, buf, n0 + c0, r0);
                            ptx::bulk_commit_group();
                        }
                    } else {
                        __syncwarp();
                        T *to = y + r0 * p.y_stride + n0 + c0;
#pragma unroll 1
                        for (int k0 = 0; k0 < WIDE; k0 += TOGETHER) {
                            T v[TOGETHER];
#pragma unroll
                            for (int k = 0; k < TOGETHER; ++k)
                                v[k] = *in_slice((k0 + k) / (WIDE / 32), (k0 + k) % (WIDE / 32) * 32 + lane);
#pragma unroll
                            for (int k = 0; k < TOGETHER; ++k) {
                                const int row = (k0 + k) / (WIDE / 32), col = (k0 + k) % (WIDE / 32) * 32 + lane;
                                if (row < high && col < wide)
                                    to[row * p.y_stride + col] = v[k];
                            }
                        }
                        __syncwarp();
                    }
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (S::PAIR)
                    ptx::mbar_arrive_cluster(ptx::map_to_rank(ptx::smem_u32(&acc_empty[a]), 0));
                else
                    ptx::mbar_arrive(&acc_empty[a]);
            }
        }
        if (lane == 0)
            ptx::bulk_wait_group<0>();
        __syncwarp();
    }
    if (p.split > 1) {
        __syncwarp();
        // the other warps' share of the epilogue's barrier, then: nobody reads this CTA's
        // sums any more
        if (warp < 2) {
            ptx::cluster_arrive_release();
            ptx::cluster_wait_acquire();
        }
        ptx::cluster_arrive_release();
        ptx::cluster_wait_acquire();
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == PRODUCER_WARP && lane == 0 && rank == 0) {
        // every load has landed before the CTA's shared memory goes away (a pair's second CTA
        // waits for the first below; where this one stopped earlier, what the other asked for
        // alone counts too)
        if constexpr (S::PAIR) {
            ptx::mbar_wait_drain(peer_done, 0, fault, limit_ns + kDefaultWaitLimitNs);
            if (ptx::mbar_try_wait_cluster(peer_done, 0))
                for (int more = static_cast<int>(*peer_total - total); more > 0; --more) {
                    ptx::mbar_arrive_expect_tx(&full[s], S::STAGE_BYTES);
                    if (issued < STAGES)
                        ++issued;
                    advance();
                }
        }
        for (; issued > 0; --issued) {
            if (s == 0) {
                s = STAGES;
                turn ^= 1;
            }
            ptx::mbar_wait_drain(&full[--s], turn, fault, kDefaultWaitLimitNs);
        }
    }
    if (warp == MMA_WARP) {
        if (lane == 0) {
            // every product has completed before tensor memory is freed
            for (int k = committed > S::ACCS ? committed - S::ACCS : 0; k < committed; ++k)
                ptx::mbar_wait_drain(&acc_full[k % S::ACCS], (k / S::ACCS) & 1, fault,
                                     kDefaultWaitLimitNs);
        }
        __syncwarp();
    }
    if (S::PAIR) {
        __syncthreads();
        ptx::cluster_arrive_release();
        ptx::cluster_wait_acquire();
    }
    if (warp == MMA_WARP) {
        ptx::tc_fence_after();
        if constexpr (S::PAIR)
            ptx::tmem_dealloc_pair(tmem, S::TMEM_COLS);
        else
            ptx::tmem_dealloc(tmem, S::TMEM_COLS);
    }
}

// ---- what TMA cannot read in place ---------------------------------------------------
// Rows of a 16-bit matrix with a pitch of whole 16 bytes, or the three parts of an fp32
// one, [part][rows][pitch].  The bits between a row's end and its pitch are not read.
constexpr int kCopyThreads = 256;

// A matrix and its copy (null: none).
template <typename T>
struct Copy {
    const T *from;
    long long stride, rows;
    unsigned short *to;
    bool vectors;  // rows start on 16-byte boundaries
};

// A thread takes eight numbers of a row, `1 << lanes` threads a row.
template <typename T>
__global__ void __launch_bounds__(kCopyThreads)
operand_kernel(const Copy<T> x, const Copy<T> w, int cols, int pitch, int lanes)
{
    ptx::griddep_launch_dependents();
    const long long rows_x = x.to ? x.rows : 0, rows = rows_x + (w.to ? w.rows : 0);
    const int lane = threadIdx.x & ((1 << lanes) - 1), down = kCopyThreads >> lanes;
    for (long long n = blockIdx.x * static_cast<long long>(down) + (threadIdx.x >> lanes); n < rows;
         n += static_cast<long long>(gridDim.x) * down) {
        const Copy<T> &m = n < rows_x ? x : w;
        const long long r = n < rows_x ? n : n - rows_x, part = m.rows * pitch;
        const T *const from = m.from + r * m.stride;
        unsigned short *const to = m.to + r * pitch;
        for (int c = lane * 8; c < cols; c += 8 << lanes) {
            T v[8];
            if (m.vectors && c + 8 <= cols) {
                constexpr int V = 16 / sizeof(T);
#pragma unroll
                for (int j = 0; j < 8; j += V)
                    *reinterpret_cast<uint4 *>(v + j) = __ldg(reinterpret_cast<const uint4 *>(from + c + j));
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = c + j < cols ? from[c + j] : T();
            }
            if constexpr (sizeof(T) == 4) {
                uint32_t o[kParts][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t parts[kParts];
                    split_pair_parts<kParts>(v[2 * j], v[2 * j + 1], parts);
                    // An infinity's are 1, 0 and itself: it meets the other number's first part,
                    // which has that number's sign, and another infinity's 1, but no part that
                    // happens to be zero.
                    const bool lo = fabsf(v[2 * j]) == CUDART_INF_F, hi = fabsf(v[2 * j + 1]) == CUDART_INF_F;
                    if (lo || hi) {
                        const uint32_t keep = (lo ? 0u : 0xffffu) | (hi ? 0u : 0xffff0000u);
                        parts[2] = (parts[2] & keep) | (bf16_pair(v[2 * j], v[2 * j + 1]) & ~keep);
                        parts[1] &= keep;
                        parts[0] = (parts[0] & keep) |
                                   (bf16_pair(copysignf(1.0f, v[2 * j]), copysignf(1.0f, v[2 * j + 1])) & ~keep);
                    }
#pragma unroll
                    for (int k = 0; k < kParts; ++k)
                        o[k][j] = parts[k];
                }
#pragma unroll
                for (int k = 0; k < kParts; ++k)
                    *reinterpret_cast<uint4 *>(to + k * part + c) =
                        make_uint4(o[k][0], o[k][1], o[k][2], o[k][3]);
            } else {
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o[j] = static_cast<uint32_t>(v[2 * j]) | static_cast<uint32_t>(v[2 * j + 1]) << 16;
                *reinterpret_cast<uint4 *>(to + c) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    }
}

template <typename T>
int copy_operands(const Copy<T> &x, const Copy<T> &w, int cols, int pitch, cudaStream_t stream)
{
    const int st = check_launch_injection("lstm_dense");
    if (st != LSTM_OK)
        return st;
    int lanes = 0;
    while (lanes < 5 && 8 << lanes < cols)
        ++lanes;
    const long long rows = (x.to ? x.rows : 0) + (w.to ? w.rows : 0);
    const long long blocks = (rows + (kCopyThreads >> lanes) - 1) / (kCopyThreads >> lanes);
    operand_kernel<T><<<static_cast<unsigned>(blocks < 152 * 8 ? blocks : 152 * 8), kCopyThreads, 0,
                        stream>>>(x, w, cols, pitch, lanes);
    return cuda_status(cudaGetLastError(), "lstm_dense launch");
}

// One operand as TMA reads it: in place, or in the workspace.
struct Operand {
    bool copied;
    int pitch;         // elements, of the copy
    size_t bytes;      // of the workspace

    Operand(const void *at, long long stride, int dtype, long long rows, int cols)
        : copied(dtype == LSTM_F32 || !rows_aligned(at, rows > 1 ? stride : 0, 2)),
          pitch((cols + 7) / 8 * 8),
          bytes(copied ? static_cast<size_t>(rows) * pitch * 2 * (dtype == LSTM_F32 ? kParts : 1) : 0)
    {
        bytes = (bytes + 255) / 256 * 256;
    }
};

// ---- launches ---------------------------------------------------------------------------
template <class S, typename T>
int launch(const CUtensorMap &a, const CUtensorMap &b, const CUtensorMap &y, DenseArgs &p, bool bf16,
           int split, bool copied, cudaStream_t stream)
{
    static SharedMemory memory;
    int st = memory.allow(dense_kernel<S, T>, S::SMEM_BYTES);
    if (st != LSTM_OK)
        return st;
    unsigned *fault = fault_word();
    if (!fault)
        return fail(LSTM_E_CUDA, "cannot resolve the device fault word");
    if ((st = check_launch_injection("lstm_dense")))
        return st;
    const int down = S::SWAP ? p.out : p.rows, along = S::SWAP ? p.rows : p.out;
    const int tiles_m = static_cast<int>((down + S::CTAS * BM - 1LL) / (S::CTAS * BM));
    const long long tiles = tiles_m * ((along + S::BN - 1LL) / S::BN);
    p.split = split;
    p.group = S::SWAP ? 1 : 12 / S::CTAS;
    // few rows: a cluster for each tile; else no more CTAs than run at once
    const long long ctas = S::SWAP || split > 1 ? tiles * split
                                                : S::CTAS * (tiles < 152 / S::CTAS ? tiles : 152 / S::CTAS);
    Dependent launch(dim3(static_cast<unsigned>(ctas)), THREADS, S::SMEM_BYTES, stream);
    launch.config.numAttrs = copied ? 1 : 0;  // (else nothing of this call comes before)
    if (S::PAIR || split > 1) {
        cudaLaunchAttribute &cluster = launch.attributes[launch.config.numAttrs++];
        cluster.id = cudaLaunchAttributeClusterDimension;
        cluster.val.clusterDim = {static_cast<unsigned>(S::PAIR ? 2 : split), 1, 1};
    }
    return cuda_status(cudaLaunchKernelEx(&launch.config, dense_kernel<S, T>, a, b, y, p,
                                          ptx::f16_idesc(BM * S::CTAS, S::BN, bf16), tiles, tiles_m, fault,
                                          kernel_test(kTestDense)),
                       "lstm_dense launch");
}

// Tiles' width and the parts of K.
struct Plan {
    bool swap;
    int width;
    int split;
    bool pair;
    // rows of a box of x and of w
    int x_rows() const { return swap ? width : BM; }
    int w_rows() const { return swap ? BM : pair ? width / 2 : width; }
};

Plan make_plan(int rows, int in, int out, int products)
{
    Plan r = {rows <= kFewRows, 0, 1, false};
    const long long kblocks = (in + BK - 1LL) / BK * products;
    long long tiles;
    if (r.swap) {
        r.width = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
        tiles = (out + BM - 1LL) / BM;
    } else {
        // What a K block of a tile takes, in cycles: the tensor core's 131 for each 16 of K at a
        // width of 256 (67 at 128, 51 at 64), or the loads, of which an SM gets 64 bytes a
        // cycle.  A pair of SMs loads half of w's rows each, 32 KB where an SM alone loads 48,
        // and so keeps its tensor cores busy.
        const long long tall = (rows + BM - 1LL) / BM;
        const auto turns = [](long long tiles, int at_once) { return (tiles + at_once - 1) / at_once; };
        const long long pairs = (rows + 2 * BM - 1LL) / (2 * BM) * ((out + 255LL) / 256);
        long long best = turns(pairs, 76) * 530;
        r.pair = true;
        r.width = 256;
        tiles = 2 * pairs;
        for (const int width : {256, 128, 64}) {
            const long long n = tall * ((out + width - 1LL) / width);
            const long long cost = turns(n, 152) * (width == 256 ? 768 : width == 128 ? 512 : 384);
            if (cost < best) {
                best = cost;
                r = {false, width, 1, false};
                tiles = n;
            }
        }
    }
    // (one CTA an SM, whose ring is deep enough to keep its share of the memory busy; clusters
    // of eight such CTAs do not all find room at a time: 128 x 4096 x 1024 takes 15 us in parts
    // of four, 23 us in parts of eight)
    while (!r.pair && r.split < 4 && tiles * r.split * 2 <= 152 && kblocks >= 8 * r.split)
        r.split *= 2;
    return r;
}

template <typename T>
int product(const CUtensorMap &x, const CUtensorMap &w, const CUtensorMap &y, DenseArgs &p,
            const Plan &plan, bool bf16, bool copied, cudaStream_t stream)
{
    if (plan.swap) {
        switch (plan.width) {
        case 16:
            return launch<Shape<16, true>, T>(w, x, y, p, bf16, plan.split, copied, stream);
        case 32:
            return launch<Shape<32, true>, T>(w, x, y, p, bf16, plan.split, copied, stream);
        default:
            return launch<Shape<64, true>, T>(w, x, y, p, bf16, plan.split, copied, stream);
        }
    }
    if (plan.pair)
        return launch<Shape<256, false, true>, T>(x, w, y, p, bf16, 1, copied, stream);
    switch (plan.width) {
    case 64:
        return launch<Shape<64, false>, T>(x, w, y, p, bf16, plan.split, copied, stream);
    case 128:
        return launch<Shape<128, false>, T>(x, w, y, p, bf16, plan.split, copied, stream);
    default:
        return launch<Shape<256, false>, T>(x, w, y, p, bf16, plan.split, copied, stream);
    }
}

CUtensorMapDataType map_type(int dtype)
{
    return dtype == LSTM_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
           : dtype == LSTM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

}  // namespace
}  // namespace lstm

using namespace lstm;

extern "C" size_t lstm_dense_workspace(const void *x, long long x_stride, const void *w,
                                       long long w_stride, int dtype, int rows, int in, int out)
{
    // (nothing for sizes that the call refuses: no memory is asked for in vain)
    if (rows <= kFewestRows || in <= 0 || out <= 0 || rows > LSTM_DENSE_MAX || in > LSTM_DENSE_MAX ||
        out > LSTM_DENSE_MAX)
        return 0;
    return Operand(x, x_stride, dtype, rows, in).bytes + Operand(w, w_stride, dtype, out, in).bytes;
}

extern "C" int lstm_dense(const void *x, long long x_stride, const void *w, long long w_stride,
                          const float *bias, int activation, const void *residual,
                          long long residual_stride, int dtype, int rows, int in, int out, void *y,
                          long long y_stride, void *workspace, size_t workspace_bytes, void *stream)
{
    const char *what = "lstm_dense";
    int st;
    if ((st = check_dtype(what, dtype)))
        return st;
    if (rows < 0 || in <= 0 || out <= 0 || activation < LSTM_ACT_NONE || activation > LSTM_ACT_SILU)
        return fail(LSTM_E_INVALID, "%s: %d rows, %d to %d columns, activation %d", what, rows, in,
                    out, activation);
    // (the kernels count the rows of all parts, and K blocks of all products, in 32 bits)
    if (rows > LSTM_DENSE_MAX || in > LSTM_DENSE_MAX || out > LSTM_DENSE_MAX)
        return fail(LSTM_E_OVERFLOW, "%s: %d rows, %d to %d columns (at most %d)", what, rows, in,
                    out, LSTM_DENSE_MAX);
    const int size = element_size(dtype);
    if ((st = check_matrix(what, "w", w, w_stride, out, in, size)) ||
        (bias && (st = check_matrix(what, "bias", bias, out, 1, out, 4))))
        return st;
    if (rows > 0 && ((st = check_matrix(what, "x", x, x_stride, rows, in, size)) ||
                     (residual && (st = check_matrix(what, "residual", residual, residual_stride,
                                                     rows, out, size))) ||
                     (st = check_matrix(what, "y", y, y_stride, rows, out, size))))
        return st;
    int device = 0;
    if ((st = op_device(w, &device)))
        return st;
    if (rows == 0)
        return LSTM_OK;
    if (rows <= kFewestRows) {
        DeviceGuard guard(device);
        if (!guard.ok)
            return fail(LSTM_E_CUDA, "cannot make device %d current", device);
        return launch_dense_few({x, w, bias, residual, y, x_stride, w_stride, residual_stride,
                                 y_stride, rows, in, out, activation}, dtype,
                                static_cast<cudaStream_t>(stream));
    }
    const Operand ox(x, x_stride, dtype, rows, in), ow(w, w_stride, dtype, out, in);
    if (ox.bytes + ow.bytes > 0 && !workspace)
        return fail(LSTM_E_INVALID, "%s: workspace is null", what);
    if (workspace_bytes < ox.bytes + ow.bytes)
        return fail(LSTM_E_LENGTH, "%s: workspace has %zu bytes, needs %zu", what, workspace_bytes,
                    ox.bytes + ow.bytes);
    if ((st = check_aligned(workspace, "workspace")))
        return st;
    DeviceGuard guard(device);
    if (!guard.ok)
        return fail(LSTM_E_CUDA, "cannot make device %d current", device);
    cudaStream_t on = static_cast<cudaStream_t>(stream);

    const Plan plan = make_plan(rows, in, out, dtype == LSTM_F32 ? kProducts : 1);
    const CUtensorMapDataType type =
        dtype == LSTM_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int parts = dtype == LSTM_F32 ? kParts : 1;
    // (both rows of `in`, and so of one pitch)
    void *const x_copy = ox.copied ? workspace : nullptr;
    void *const w_copy = ow.copied ? static_cast<char *>(workspace) + ox.bytes : nullptr;
    if (ox.copied || ow.copied) {
        const auto copy = [&](auto type) {
            using T = decltype(type);
            const auto one = [&](const void *from, long long stride, long long n, void *to) {
                return Copy<T>{static_cast<const T *>(from), stride, n, static_cast<unsigned short *>(to),
                               rows_aligned(from, n > 1 ? stride : 0, sizeof(T))};
            };
            return copy_operands<T>(one(x, x_stride, rows, x_copy), one(w, w_stride, out, w_copy), in,
                                    ox.pitch, on);
        };
        st = dtype == LSTM_F32 ? copy(0.0f) : copy(static_cast<unsigned short>(0));
        if (st != LSTM_OK)
            return st;
    }
    const auto map = [&](CUtensorMap *m, const void *copy, const void *at, long long stride, long long n,
                         int box_rows) {
        const long long own = ox.pitch;  // (of one row the stride says nothing)
        return encode_box_map(m, type, copy ? copy : at, n * parts, in,
                              (copy || n == 1 ? own : stride) * 2, box_rows);
    };
    CUtensorMap x_map, w_map, y_map = {};
    if ((st = map(&x_map, x_copy, x, x_stride, rows, plan.x_rows())) ||
        (st = map(&w_map, w_copy, w, w_stride, out, plan.w_rows())))
        return st;
    DenseArgs p = {x, w, x_stride, w_stride, bias, residual, y, residual_stride, y_stride, rows, in,
                   out, activation, dtype == LSTM_F32 ? kProducts : 1, 1, false, false, false, 1};
    p.whole = rows_aligned(bias, 0, 4);
    // (whole vectors: what lies behind a row's last numbers is not read)
    p.vectors = residual && rows_aligned(residual, rows > 1 ? residual_stride : 0, size) &&
                out * size % 16 == 0;
    p.store_boxes = !plan.swap && rows_aligned(y, y_stride, size);
    if (p.store_boxes &&
        (st = encode_box_map(&y_map, map_type(dtype), y, rows, out, y_stride * size, 32)))
        return st;
    LSTM_WITH_TYPE(dtype, T,
                   return product<T>(x_map, w_map, y_map, p, plan, dtype != LSTM_F16,
                                     ox.copied || ow.copied, on));
}
