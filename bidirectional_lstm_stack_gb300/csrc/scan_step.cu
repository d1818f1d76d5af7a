// The selective scan's next token of every sequence.
//
// Memory-bound: the states are read and written once, 8 bytes a state against
// some eight operations.  256 sequences of 4096 channels x 16 states in a pool of
// 300: 26 us, 5.5 TB/s, 80 % of the card's copy rate (tiles' kernel; the other one
// 38 us).
#include "scan.cuh"

namespace lstm {
namespace {

constexpr int kThreads = 128;

constexpr int kStages = 4;  // sequences whose states are on their way to a thread

// The general kernel.  A thread owns four states of a channel (16 bytes, so
// that a warp's accesses are whole consecutive lines) and L lanes a channel.  It
// keeps its place in the states and goes through the sequences s0,
// s0 + gridDim.y, ...: a, skip and the bias are loaded once, the next states
// come asynchronously to a ring in shared memory, each thread's own, and the
// next inputs to registers.  grid (channel blocks, sequences at a time).
template <typename T, int L, bool WIDE>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(ScanArgs p)
{
    constexpr int kAcross = kThreads / L;  // channels of a block
    __shared__ __align__(16) float ring[kStages][kThreads][4];
    const int d0 = blockIdx.x * kAcross + threadIdx.x / L;
    const bool live = d0 < p.channels;
    const int d = live ? d0 : 0;
    const int n0 = threadIdx.x % L * 4;
    const int group = p.groups > 1 ? d / (p.channels / p.groups) : 0;
    const int step = gridDim.y;
    const long long at = static_cast<long long>(d) * p.states + n0;
    const auto in = [&](int n) { return live && n0 + n < p.states; };
    const auto place = [&](int slot) {
        return p.state + static_cast<long long>(slot) * p.channels * p.states + at;
    };
    const auto fetch = [&](int s, int slot, float (&to)[4]) {
        if (s < p.seq.count && slot >= 0) {
            const float *from = place(slot);
            if (WIDE) {
                ptx::cp_async_16(ptx::smem_u32(to), in(0) ? from : p.state, in(0) ? 16 : 0);
            } else {
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    ptx::cp_async_4(ptx::smem_u32(to + n), in(n) ? from + n : p.state,
                                    in(n) ? 4 : 0);
            }
        } else {
            *reinterpret_cast<float4 *>(to) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        ptx::cp_async_commit();
    };
    const auto slot_of = [&](int s) { return s < p.seq.count ? sequence_slot(p.slots, s) : -1; };
    struct Inputs {
        T u, dt, z, b[4], c[4];
    };
    const auto read = [&](int s, Inputs &x) {
        if (s >= p.seq.count)
            return;
        x.u = static_cast<const T *>(p.u)[s * p.u_stride + d];
        x.dt = static_cast<const T *>(p.dt)[s * p.dt_stride + d];
        if (p.z)
            x.z = static_cast<const T *>(p.z)[s * p.z_stride + d];
        const T *b = static_cast<const T *>(p.b) + s * p.b_stride + group * p.states + n0;
        const T *c = static_cast<const T *>(p.c) + s * p.c_stride + group * p.states + n0;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            x.b[n] = n0 + n < p.states ? b[n] : Elem<T>::put(0.0f);
            x.c[n] = n0 + n < p.states ? c[n] : Elem<T>::put(0.0f);
        }
    };

    const int s0 = blockIdx.y;
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k)
        fetch(s0 + k * step, slot_of(s0 + k * step), ring[k][threadIdx.x]);
    int next_slot = slot_of(s0 + (kStages - 1) * step);
    Inputs next;
    read(s0, next);
    float a[4];
#pragma unroll
    for (int n = 0; n < 4; ++n)
        a[n] = in(n) ? kLog2e * __ldg(p.a + at + n) : 0.0f;
    const float skip = p.skip ? __ldg(p.skip + d) : 0.0f;
    const float dt_bias = p.dt_bias ? __ldg(p.dt_bias + d) : 0.0f;
    int k = 0;
    for (int s = s0; s < p.seq.count; s += step, ++k) {
        fetch(s + (kStages - 1) * step, next_slot, ring[(k + kStages - 1) % kStages][threadIdx.x]);
        next_slot = slot_of(s + kStages * step);
        const int slot = slot_of(s);
        const Inputs x = next;
        read(s + step, next);
        float st = Elem<T>::get(x.dt) + dt_bias;
        if (p.softplus) {
            Pair v[1] = {make_pair(st, st)};
            softplus_pairs(v);
            st = split_pair(v[0]).x;
        }
        const float ut = Elem<T>::get(x.u), su = st * ut;
        ptx::cp_async_wait<kStages - 1>();
        float h[4], v = 0.0f;
        *reinterpret_cast<float4 *>(h) =
            *reinterpret_cast<const float4 *>(ring[k % kStages][threadIdx.x]);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            h[n] = fmaf(ex2(st * a[n]), h[n], su * Elem<T>::get(x.b[n]));
            // (places beyond the states have no part in the output: an infinite
            // input makes NaN of their zeros)
            if (WIDE || n0 + n < p.states)
                v = fmaf(h[n], Elem<T>::get(x.c[n]), v);
        }
        if (WIDE && n0 >= p.states)
            v = 0.0f;
        if (slot >= 0) {
            float *to = place(slot);
            if (WIDE) {
                if (in(0))
                    *reinterpret_cast<float4 *>(to) = *reinterpret_cast<float4 *>(h);
            } else {
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    if (in(n))
                        to[n] = h[n];
            }
        }
#pragma unroll
        for (int m = 1; m < L; m <<= 1)
            v += __shfl_xor_sync(0xffffffffu, v, m);
        if (live && n0 == 0) {
            if (p.skip)  // (0 times an infinity is no 0)
                v = fmaf(skip, ut, v);
            if (p.z)
                v *= silu(Elem<T>::get(x.z));
            static_cast<T *>(p.y)[s * p.y_stride + d] = Elem<T>::put(v);
        }
    }
}

// The same for many sequences whose states come in whole tiles: the states of
// a block's channels are one run of memory, copied to and from a ring of tiles
// by the TMA engine, and a thread works on NS states of a channel in one go (L
// lanes a channel: states = NS * L), so that what a channel needs once is
// computed by L threads instead of by one for every four states.  Threads
// stand NS states apart, so each starts its tile reads at another quad (they
// would meet in the same banks otherwise).
constexpr int kTiles = 4;

template <typename T, int NS, int L>
__global__ void __launch_bounds__(kThreads) scan_step_tiles_kernel(ScanArgs p, unsigned *fault,
                                                                     KernelTest test)
{
    constexpr int kAcross = kThreads / L;  // channels of a block
    constexpr int kQuads = NS / 4, kStates = NS * L;
    constexpr int kApart = kQuads > 1 ? 8 / kQuads : 1;  // threads that share a first quad
    __shared__ __align__(128) float tiles[kTiles][kThreads * NS];
    __shared__ __align__(16) float sb[2][kStates], sc[2][kStates];
    __shared__ uint64_t full[kTiles];
    __shared__ volatile int abort;
    const int c0 = blockIdx.x * kAcross;
    const int here = min(kAcross, p.channels - c0);
    const uint32_t bytes = here * kStates * 4;
    const int ch = threadIdx.x / L;
    const bool live = ch < here;
    const int d = c0 + (live ? ch : 0);
    const int n0 = threadIdx.x % L * NS;
    const int first = threadIdx.x / kApart % kQuads;  // quad that this thread starts with
    const auto quad = [&](int q) { return (q + first) % kQuads * 4; };
    const int group = p.groups > 1 ? c0 / (p.channels / p.groups) : 0;
    const int step = gridDim.y, s0 = blockIdx.y;
    const auto slot_of = [&](int s) { return s < p.seq.count ? sequence_slot(p.slots, s) : -1; };
    const auto place = [&](int slot) {
        return p.state + (static_cast<long long>(slot) * p.channels + c0) * kStates;
    };
    int fetched = 0;
    const auto fetch = [&](int k, int slot) {  // by one thread
        if (test.withhold)
            return;
        fetched = k + 1;
        if (slot >= 0) {
            ptx::mbar_arrive_expect_tx(&full[k % kTiles], bytes);
            ptx::bulk_load(tiles[k % kTiles], place(slot), bytes, &full[k % kTiles]);
        } else {
            ptx::mbar_arrive(&full[k % kTiles]);
        }
    };
    if (threadIdx.x == 0) {
        for (int k = 0; k < kTiles; ++k)
            ptx::mbar_init(&full[k], 1);
        abort = 0;
        ptx::fence_mbar_init();
        for (int k = 0; k < kTiles - 2; ++k)
            if (s0 + k * step < p.seq.count)
                fetch(k, slot_of(s0 + k * step));
    }
    struct Inputs {
        T u, dt, z, b, c;
    };
    const T *u = static_cast<const T *>(p.u) + s0 * p.u_stride + d;
    const T *dt = static_cast<const T *>(p.dt) + s0 * p.dt_stride + d;
    const T *z = p.z ? static_cast<const T *>(p.z) + s0 * p.z_stride + d : nullptr;
    const T *b = static_cast<const T *>(p.b) + s0 * p.b_stride + group * kStates + threadIdx.x;
    const T *c = static_cast<const T *>(p.c) + s0 * p.c_stride + group * kStates + threadIdx.x;
    T *y = static_cast<T *>(p.y) + s0 * p.y_stride + d;
    const long long u_step = step * p.u_stride, dt_step = step * p.dt_stride,
                    z_step = step * p.z_stride, b_step = step * p.b_stride,
                    c_step = step * p.c_stride, y_step = step * p.y_stride;
    const auto read_row = [&](Inputs &x) {
        x.u = *u;
        x.dt = *dt;
        if (z)
            x.z = *z;
        u += u_step;
        dt += dt_step;
        if (z)
            z += z_step;
    };
    const auto read_shared = [&](Inputs &x) {
        if (threadIdx.x < kStates) {
            x.b = *b;
            x.c = *c;
        }
        b += b_step;
        c += c_step;
    };
    const auto settle = [&](const Inputs &x, int at) {
        if (threadIdx.x < kStates) {
            sb[at][threadIdx.x] = Elem<T>::get(x.b);
            sc[at][threadIdx.x] = Elem<T>::get(x.c);
        }
    };
    Inputs next, shared;
    read_row(next);
    read_shared(shared);
    float a[NS];
#pragma unroll
    for (int q = 0; q < kQuads; ++q) {
        load_weights<4>(p.a + static_cast<long long>(d) * kStates + n0 + quad(q),
                        reinterpret_cast<float(&)[4]>(a[4 * q]));
#pragma unroll
        for (int n = 0; n < 4; ++n)
            a[4 * q + n] *= kLog2e;
    }
    const float skip = p.skip ? __ldg(p.skip + d) : 0.0f;
    const float dt_bias = p.dt_bias ? __ldg(p.dt_bias + d) : 0.0f;
    settle(shared, 0);
    __syncthreads();
    int k = 0;
    for (int s = s0; s < p.seq.count; s += step, ++k) {
        // the tile that is fetched now was written back two turns ago
        if (threadIdx.x == 0 && s + (kTiles - 2) * step < p.seq.count) {
            ptx::bulk_wait_group_read<1>();
            fetch(k + kTiles - 2, slot_of(s + (kTiles - 2) * step));
        }
        const Inputs x = next;
        const bool more = s + step < p.seq.count;
        if (more) {
            read_row(next);
            read_shared(shared);
        }
        const int slot = slot_of(s);
        Pair v[1] = {make_pair(Elem<T>::get(x.dt) + dt_bias, 0.0f)};
        const float plain = split_pair(v[0]).x;
        if (p.softplus)
            softplus_pairs(v);
        const float st = p.softplus ? split_pair(v[0]).x : plain;
        const float ut = Elem<T>::get(x.u), su = st * ut;
        float *tile = tiles[k % kTiles] + threadIdx.x * NS;
        if (!ptx::mbar_wait_bounded(&full[k % kTiles], k / kTiles & 1, &abort, fault, kFaultScanStep,
                                    test.wait_limit_ns))
            break;
        float out = 0.0f;
#pragma unroll
        for (int q = 0; q < kQuads; ++q) {
            float4 h = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (slot >= 0)
                h = *reinterpret_cast<const float4 *>(tile + quad(q));
            const float4 bn = *reinterpret_cast<const float4 *>(&sb[k & 1][n0 + quad(q)]);
            const float4 cn = *reinterpret_cast<const float4 *>(&sc[k & 1][n0 + quad(q)]);
            h.x = fmaf(ex2(st * a[4 * q]), h.x, su * bn.x);
            h.y = fmaf(ex2(st * a[4 * q + 1]), h.y, su * bn.y);
            h.z = fmaf(ex2(st * a[4 * q + 2]), h.z, su * bn.z);
            h.w = fmaf(ex2(st * a[4 * q + 3]), h.w, su * bn.w);
            out = fmaf(h.x, cn.x, out);
            out = fmaf(h.y, cn.y, out);
            out = fmaf(h.z, cn.z, out);
            out = fmaf(h.w, cn.w, out);
            *reinterpret_cast<float4 *>(tile + quad(q)) = h;
        }
#pragma unroll
        for (int m = 1; m < L; m <<= 1)
            out += __shfl_xor_sync(0xffffffffu, out, m);
        if (live && n0 == 0) {
            if (p.skip)
                out = fmaf(skip, ut, out);
            if (z)
                out *= silu(Elem<T>::get(x.z));
            *y = Elem<T>::put(out);
        }
        y += y_step;
        if (more)
            settle(shared, (k + 1) & 1);
        ptx::fence_proxy_async_smem();
        __syncthreads();
        if (threadIdx.x == 0) {
            if (slot >= 0)
                ptx::bulk_store(place(slot), tiles[k % kTiles], bytes);
            ptx::bulk_commit_group();
        }
    }
    if (threadIdx.x == 0) {
        // after a wait that ran out: copies that were asked for may still land
        for (; abort && k < fetched; ++k)
            ptx::mbar_wait_drain(&full[k % kTiles], k / kTiles & 1, fault, test.wait_limit_ns);
        ptx::bulk_wait_group<0>();
    }
}

template <typename T, int NS, int L>
int launch_tiles(const ScanArgs &p, cudaStream_t stream)
{
    unsigned *fault = fault_word();
    if (!fault)
        return fail(LSTM_E_CUDA, "cannot resolve the device fault word");
    const int st = check_launch_injection("lstm_selective_scan_step");
    if (st != LSTM_OK)
        return st;
    const long long blocks = (p.channels + kThreads / L - 1) / (kThreads / L);
    long long rows = (152 * 4 + blocks - 1) / blocks;
    rows = rows < p.seq.count ? rows : p.seq.count;
    scan_step_tiles_kernel<T, NS, L>
        <<<dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(rows)), kThreads, 0, stream>>>(
            p, fault, kernel_test(kTestScanStep));
    return cuda_status(cudaGetLastError(), "lstm_selective_scan_step launch");
}

// Whether the tiles' kernel takes the call (for 4, 8, .. 128 states; it is not
// instantiated for other counts, which take the general kernel: 256 sequences x
// 4096 channels x 24 states 77 us, x 48 156 us, where their bytes take 30 and
// 59): states of a channel block are one run of whole 16-byte units, no block
// spans two groups, and there are enough states for the ring to pay (8 sequences
// x 2048 channels x 16 states: 3.0 us with it, 2.8 without; 32 sequences: 3.7 and
// 4.4).
bool takes_tiles(const ScanArgs &p, int lanes)
{
    const int across = kThreads / lanes;
    return p.state && rows_aligned(p.state, 4, 4) && (reinterpret_cast<uintptr_t>(p.a) & 15) == 0 &&
           (p.groups == 1 || p.channels / p.groups % across == 0) &&
           static_cast<long long>(p.seq.count) * p.channels * p.states >= 1 << 19;
}

template <typename T, int L>
int launch_step(const ScanArgs &p, cudaStream_t stream)
{
    const long long blocks = (p.channels + kThreads / L - 1) / (kThreads / L);
    // as many sequences at a time as fill the SMs with blocks
    long long rows = (152 * 8 + blocks - 1) / blocks;
    rows = rows < p.seq.count ? rows : p.seq.count;
    rows = rows < 65535 ? rows : 65535;
    const int st = check_launch_injection("lstm_selective_scan_step");
    if (st != LSTM_OK)
        return st;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(rows));
    // whole quads where each channel's states start on a 16-byte boundary
    if (p.states % 4 == 0 && rows_aligned(p.state, p.states, 4))
        scan_step_kernel<T, L, true><<<grid, kThreads, 0, stream>>>(p);
    else
        scan_step_kernel<T, L, false><<<grid, kThreads, 0, stream>>>(p);
    return cuda_status(cudaGetLastError(), "lstm_selective_scan_step launch");
}

template <typename T>
int launch_typed(const ScanArgs &p, cudaStream_t stream)
{
    switch (p.states) {
    case 4:
        if (takes_tiles(p, 1))
            return launch_tiles<T, 4, 1>(p, stream);
        break;
    case 8:
        if (takes_tiles(p, 1))
            return launch_tiles<T, 8, 1>(p, stream);
        break;
    case 16:
        if (takes_tiles(p, 1))
            return launch_tiles<T, 16, 1>(p, stream);
        break;
    case 32:
        if (takes_tiles(p, 2))
            return launch_tiles<T, 16, 2>(p, stream);
        break;
    case 64:
        if (takes_tiles(p, 4))
            return launch_tiles<T, 16, 4>(p, stream);
        break;
    case 128:
        if (takes_tiles(p, 8))
            return launch_tiles<T, 16, 8>(p, stream);
        break;
    }
    if (p.states <= 4)
        return launch_step<T, 1>(p, stream);
    if (p.states <= 8)
        return launch_step<T, 2>(p, stream);
    if (p.states <= 16)
        return launch_step<T, 4>(p, stream);
    if (p.states <= 32)
        return launch_step<T, 8>(p, stream);
    if (p.states <= 64)
        return launch_step<T, 16>(p, stream);
    return launch_step<T, 32>(p, stream);
}

}  // namespace

int launch_scan_step(const ScanArgs &p, int dtype, cudaStream_t stream)
{
    LSTM_WITH_TYPE(dtype, T, return launch_typed<T>(p, stream));
}

}  // namespace lstm
