// scan.cu -- the gated linear recurrence h_t = alpha_t h_{t-1} + w_t x_t per
// channel: forward, backward and single step.
//
// One pass over the data.  A CTA takes 64 channels and 64 tokens at a time: its four
// warps hold 16 tokens each in registers (two channels a lane), reduce them to the map
// h -> A h + H of their span, and compose the maps of the spans before theirs through
// shared memory; then every warp knows the state it starts from and runs its tokens.
// When channels alone do not fill the device, a cluster of up to eight CTAs takes
// consecutive spans of 64 tokens of the same channels and exchanges its maps through
// distributed shared memory.  The walk over the sequence carries the state in registers,
// and the next spans' tiles arrive by TMA meanwhile (two CTAs an SM; channel counts that
// TMA cannot address, whose rows are not a multiple of 16 bytes, take plain loads).
// Bound by HBM: 8 x 4096 x 2048 bf16 forward 115 us (5.9 TB/s), backward 213 us (5.8);
// 1 x 65536 x 2048 forward 245 us (5.5: clusters of 8, whose exchange is on the walk).
//
// Backward: the same with time reversed, on c_t = alpha_t g_t (the gradient that leaves a
// token towards the past): c -> A c + G.  h_{t-1} comes from the forward's checkpoints,
// one per 16 tokens, recomputed in fp32.
#include <cooperative_groups.h>
#include <cuda.h>

#include <type_traits>

#include "common.cuh"
#include "hybrid.h"
#include "launch.h"
#include "packed.cuh"
#include "sm100.cuh"

namespace gdn2 {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kTok = kScanBlock;          // tokens of a warp
constexpr int kSpan = kWarps * kTok;      // tokens of a CTA
constexpr int kChan = 64;                 // channels of a CTA
constexpr int kMaxCluster = 8;

// The pair of channels c, c + 1 of a row; 0 outside [0, C).
template <bool EVEN, typename E>
__device__ __forceinline__ f2 load_pair(const E *row, int c, int C)
{
    if constexpr (EVEN) {
        if (c >= C) return 0;
        alignas(8) E e[2];
        if constexpr (sizeof(E) == 4) *reinterpret_cast<float2 *>(e) = __ldg(reinterpret_cast<const float2 *>(row + c));
        else *reinterpret_cast<uint32_t *>(e) = __ldg(reinterpret_cast<const uint32_t *>(row + c));
        return pair_of(e);
    } else {
        return pack2(c < C ? to_f32(row[c]) : 0.f, c + 1 < C ? to_f32(row[c + 1]) : 0.f);
    }
}
// The pair of a state that the kernel's own result may overwrite (not through the read-only
// path, whose loads may be moved over a barrier).
template <bool EVEN>
__device__ __forceinline__ f2 load_state(const float *row, int c, int C)
{
    if constexpr (EVEN) {
        if (c >= C) return 0;
        const float2 v = *reinterpret_cast<const float2 *>(row + c);
        return pack2(v.x, v.y);
    } else {
        return load_pair<EVEN>(row, c, C);
    }
}
template <bool EVEN, typename E>
__device__ __forceinline__ void store_pair(E *row, int c, int C, f2 v)
{
    const float2 u = unpack2(v);
    if constexpr (EVEN) {
        if (c >= C) return;
        if constexpr (sizeof(E) == 4) *reinterpret_cast<float2 *>(row + c) = u;
        else *reinterpret_cast<uint32_t *>(row + c) = bf16_pair(v);
    } else {
        if (c < C) row[c] = from_f32<E>(u.x);
        if (c + 1 < C) row[c + 1] = from_f32<E>(u.y);
    }
}
__device__ __forceinline__ f2 exp_pair(f2 v)
{
    const float2 u = unpack2(v);
    return pack2(expf(u.x), expf(u.y));
}

// Maps s -> A s + H of spans in order: of a CTA's warps, and of a cluster's CTAs.
struct Maps {
    ulonglong2 warp[2][kWarps][32];       // [parity][warp][lane] {A, H}
    ulonglong2 cta[2][kMaxCluster][32];   // [parity][CTA][lane]
    uint64_t landed[2];                   // [parity]: every CTA's map is here
};
// From this warp's map and the running state: the state `in` entering its span; `state`
// becomes the one behind the whole cluster's span.  `order` is the warp's (or the CTA's)
// position along the walk.  `ok`: this thread's waits so far; false for the whole CTA, which
// then ends its walk, if one of them gave up before this step (one that gives up in this step
// leaves ok false in its thread).
template <bool CL>
__device__ __forceinline__ bool enter_span(Maps &m, int step, int order, f2 A, f2 H, f2 &state, f2 &in, bool &ok, unsigned int *err)
{
    const int parity = step & 1;
    const int lane = threadIdx.x & 31;
    m.warp[parity][order][lane] = make_ulonglong2(A, H);
    ok = __syncthreads_and(ok);
    if (!ok) return false;
    f2 pa = both(1.f), ph = 0, ta = both(1.f), th = 0;  // before this warp, and in all
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w == order) pa = ta, ph = th;
        const ulonglong2 v = m.warp[parity][w][lane];
        ta = mul2(v.x, ta);
        th = fma2(v.x, th, v.y);
    }
    in = state;
    if constexpr (CL) {
        // each CTA sends its map to all and waits for theirs: 16 bytes a lane that signal the
        // receiver's barrier (1 x 65536 x 2048 bf16: 245 us, against 332 us with a barrier of
        // the whole cluster).  A CTA that sends for step k + 2 has this CTA's map of k + 1,
        // sent when its k was read.
        cg::cluster_group cluster = cg::this_cluster();
        const int size = cluster.num_blocks(), rank = cluster.block_rank();
        if (threadIdx.x == 0) sm100::mbar_arrive_expect_tx(m.landed + parity, size * 512);
        for (int p = order; p < size; p += kWarps)
            sm100::st_async_16(sm100::peer_smem(&m.cta[parity][rank][lane], p), make_ulonglong2(ta, th),
                               sm100::peer_smem(m.landed + parity, p));
        ok = sm100::mbar_wait(m.landed + parity, (step >> 1) & 1, err);
        f2 s = state;
        for (int r = 0; r < size; ++r) {
            if (r == rank) in = s;
            const ulonglong2 v = m.cta[parity][r][lane];
            s = fma2(v.x, s, v.y);
        }
        state = s;
    } else {
        state = fma2(ta, state, th);
    }
    in = fma2(pa, in, ph);
    return true;
}

// Where a CTA works: channels, batch, and its place among the CTAs of its span.
struct Place {
    int c, b, rank, size;
    __device__ __forceinline__ Place(int csize)
        : c((int)(blockIdx.x / csize) * kChan + 2 * (threadIdx.x & 31)), b(blockIdx.y), rank(blockIdx.x % csize), size(csize) {}
};

// How a kernel gets its rows: element by element, pairs, or tiles by TMA.
enum Source { kOdd, kEven, kTile };

// One span's tiles in shared memory: log_alpha, then x, w (and dy), [64 tokens][64 channels].
template <typename E, int NE>
struct Stage {
    static constexpr int LA = 0, TILE = kSpan * kChan;
    static constexpr int BYTES = TILE * 4 + NE * TILE * (int)sizeof(E);
    static constexpr int COUNT = NE == 2 ? (sizeof(E) == 2 ? 3 : 2) : (sizeof(E) == 2 ? 2 : 1);  // stages of a CTA
    static constexpr int el(int k) { return TILE * 4 + k * TILE * (int)sizeof(E); }
};
struct SpanMaps {
    CUtensorMap la, e[3];
};
template <typename E, int NE>
__device__ __forceinline__ void fetch_span(uint8_t *st, const SpanMaps &m, uint64_t *bar, int c, long long row)
{
    using S = Stage<E, NE>;
    sm100::mbar_arrive_expect_tx(bar, S::BYTES);
    sm100::tma_load_2d(st + S::LA, &m.la, bar, c, (int)row);
#pragma unroll
    for (int k = 0; k < NE; ++k) sm100::tma_load_2d(st + S::el(k), &m.e[k], bar, c, (int)row);
}

// (one thread) waits for the stages that hold the next `left` spans, at most all of them.
template <int COUNT>
__device__ __forceinline__ void drain(uint64_t *full, int st, uint32_t ph, long long left, unsigned int *err)
{
    for (int i = 0; i < COUNT && i < left; ++i) {
        (void)sm100::mbar_wait(full + st, ph, err);
        if (++st == COUNT) st = 0, ph ^= 1;
    }
}

// Token t (of the warp's 16) of a tensor: from the stage, or from memory.
template <Source SRC, typename T>
__device__ __forceinline__ f2 take(const uint8_t *tile, const T *row, int warp_row, int t, int c, int C)
{
    if constexpr (SRC == kTile) return pair_of(reinterpret_cast<const T *>(tile) + (warp_row + t) * kChan + 2 * (threadIdx.x & 31));
    else return load_pair<SRC == kEven>(row + (long long)t * C, c, C);
}

template <typename E, Source SRC, bool CL>
__global__ void __launch_bounds__(kThreads, 2)
scan_fwd_kernel(const ScanArgs a, int csize, const __grid_constant__ SpanMaps tm)
{
    using S = Stage<E, 2>;
    constexpr bool EVEN = SRC != kOdd;
    extern __shared__ __align__(128) uint8_t dyn[];
    __shared__ Maps maps;
    __shared__ __align__(8) uint64_t full[S::COUNT];
    const Place pl(csize);
    const int warp = threadIdx.x >> 5, c = pl.c, c_cta = (int)(blockIdx.x / csize) * kChan;
    const long long seq = (long long)pl.b * a.T, step = (long long)kSpan * pl.size;
    const int nblk = (a.T - 1) / kTok + 1;
    if (SRC == kTile && threadIdx.x == 0) {
        for (int i = 0; i < S::COUNT; ++i) sm100::mbar_init(full + i, 1);
        sm100::fence_mbar_init();
        for (int i = 0; i < S::COUNT; ++i)
            if (i * step < a.T) fetch_span<E, 2>(dyn + i * S::BYTES, tm, full + i, c_cta, seq + i * step + pl.rank * kSpan);
    }
    if (CL && threadIdx.x < 2) {
        sm100::mbar_init(maps.landed + threadIdx.x, 1);
        sm100::fence_mbar_init();
    }
    f2 state = a.h0 ? load_state<EVEN>(a.h0 + (long long)pl.b * a.C, c, a.C) : 0;
    __syncthreads();
    if constexpr (CL) cg::this_cluster().sync();  // every CTA has started (and read h0, which h_T may alias)
    int k = 0, st = 0;
    uint32_t ph = 0;
    bool ok = true;
    long long s0 = 0;
    for (; s0 < a.T; s0 += step, ++k) {
        const long long t0 = s0 + pl.rank * kSpan + warp * kTok;
        const int live = t0 >= a.T ? 0 : a.T - t0 < kTok ? (int)(a.T - t0) : kTok;
        const long long row = (seq + t0) * a.C;
        const uint8_t *tile = dyn + st * S::BYTES;
        if (SRC == kTile) ok = sm100::mbar_wait(full + st, ph, a.err) && ok;
        f2 al[kTok], u[kTok], A = both(1.f), H = 0;
        auto gather = [&](auto whole) {
#pragma unroll
            for (int t = 0; t < kTok; ++t) {
                const bool on = decltype(whole)::value || t < live;
                al[t] = on ? take<SRC>(tile + S::LA, a.la + row, warp * kTok, t, c, a.C) : 0;
                u[t] = on ? mul2(take<SRC>(tile + S::el(0), static_cast<const E *>(a.x) + row, warp * kTok, t, c, a.C),
                                 take<SRC>(tile + S::el(1), static_cast<const E *>(a.w) + row, warp * kTok, t, c, a.C)) : 0;
            }
        };
        if (live == kTok) gather(std::true_type());
        else gather(std::false_type());
#pragma unroll
        for (int t = 0; t < kTok; ++t) {
            al[t] = exp_pair(al[t]);
            A = mul2(al[t], A);
            H = fma2(al[t], H, u[t]);
        }
        f2 h;
        if (!enter_span<CL>(maps, k, warp, A, H, state, h, ok, a.err)) break;
        if (SRC == kTile) {  // (behind the barrier of enter_span: every warp has its tokens in registers)
            if (threadIdx.x == 0 && s0 + S::COUNT * step < a.T)
                fetch_span<E, 2>(dyn + st * S::BYTES, tm, full + st, c_cta, seq + s0 + S::COUNT * step + pl.rank * kSpan);
            if (++st == S::COUNT) st = 0, ph ^= 1;
        }
        if (live > 0 && a.ckpt) store_pair<EVEN>(a.ckpt + ((long long)pl.b * nblk + t0 / kTok) * a.C, c, a.C, h);
        E *y = static_cast<E *>(a.y) + row;
#pragma unroll
        for (int t = 0; t < kTok; ++t) {
            h = fma2(al[t], h, u[t]);
            if (t < live) store_pair<EVEN>(y, c, a.C, h);
            y += a.C;
        }
    }
    if (__builtin_expect(!ok, 0)) {
        // a wait gave up: the tiles asked for have landed, and no map is on its way, before the CTA ends
        if (SRC == kTile && threadIdx.x == 0) drain<S::COUNT>(full, st, ph, s0 < a.T ? (a.T - 1 - s0) / step + 1 : 0, a.err);
        if (CL) sm100::leave_cluster();
        return;
    }
    if (a.h_T && warp == 0 && pl.rank == 0) store_pair<EVEN>(a.h_T + (long long)pl.b * a.C, c, a.C, state);
}

template <typename E, Source SRC, bool CL>
__global__ void __launch_bounds__(kThreads, 2)
scan_bwd_kernel(const ScanArgs a, int csize, const __grid_constant__ SpanMaps tm)
{
    using S = Stage<E, 3>;
    constexpr bool EVEN = SRC != kOdd;
    extern __shared__ __align__(128) uint8_t dyn[];
    __shared__ Maps maps;
    __shared__ __align__(8) uint64_t full[S::COUNT], empty[S::COUNT];
    const Place pl(csize);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = pl.c, c_cta = (int)(blockIdx.x / csize) * kChan;
    const long long seq = (long long)pl.b * a.T, step = (long long)kSpan * pl.size, spans = (a.T + step - 1) / step;
    const int nblk = (a.T - 1) / kTok + 1;
    // along the walk the last tokens come first: rank 0 and warp 0 take the latest
    auto first_token = [&](long long sp) { return sp * step + (pl.size - 1 - pl.rank) * kSpan; };
    if (SRC == kTile && threadIdx.x == 0) {
        for (int i = 0; i < S::COUNT; ++i) {
            sm100::mbar_init(full + i, 1);
            sm100::mbar_init(empty + i, kWarps);
        }
        sm100::fence_mbar_init();
        for (int i = 0; i < S::COUNT && i < spans; ++i)
            fetch_span<E, 3>(dyn + i * S::BYTES, tm, full + i, c_cta, seq + first_token(spans - 1 - i));
    }
    if (CL && threadIdx.x < 2) {
        sm100::mbar_init(maps.landed + threadIdx.x, 1);
        sm100::fence_mbar_init();
    }
    f2 state = a.dh_T ? load_state<EVEN>(a.dh_T + (long long)pl.b * a.C, c, a.C) : 0;
    __syncthreads();
    if constexpr (CL) cg::this_cluster().sync();  // every CTA has started (and read dh_T, which dh0 may alias)
    int k = 0, st = 0;
    uint32_t ph = 0;
    bool ok = true;
    long long sp = spans - 1;
    for (; sp >= 0; --sp, ++k) {
        const int wrow = (kWarps - 1 - warp) * kTok;
        const long long t0 = first_token(sp) + wrow;
        const int live = t0 >= a.T ? 0 : a.T - t0 < kTok ? (int)(a.T - t0) : kTok;
        const long long row = (seq + t0) * a.C;
        const E *x = static_cast<const E *>(a.x) + row, *w = static_cast<const E *>(a.w) + row, *dy = static_cast<const E *>(a.dy) + row;
        const uint8_t *tile = dyn + st * S::BYTES;
        f2 h = live ? load_pair<EVEN>(a.ckpt + ((long long)pl.b * nblk + t0 / kTok) * a.C, c, a.C) : 0;
        if (SRC == kTile) ok = sm100::mbar_wait(full + st, ph, a.err) && ok;
        // x, w and dy are taken twice (from the stage, or from cache): kept in registers they
        // would halve the warps of an SM
        auto get = [&](int k, const E *p, int t) { return take<SRC>(tile + S::el(k), p, wrow, t, c, a.C); };
        f2 al[kTok], hp[kTok], A = both(1.f), G = 0;
        auto gather = [&](auto whole) {
#pragma unroll
            for (int t = 0; t < kTok; ++t) {
                const bool on = decltype(whole)::value || t < live;
                al[t] = on ? exp_pair(take<SRC>(tile + S::LA, a.la + row, wrow, t, c, a.C)) : both(1.f);
                hp[t] = h;
                if (on) h = fma2(al[t], h, mul2(get(0, x, t), get(1, w, t)));
            }
#pragma unroll
            for (int t = kTok - 1; t >= 0; --t) {
                const bool on = decltype(whole)::value || t < live;
                A = mul2(al[t], A);
                G = mul2(al[t], on ? add2(get(2, dy, t), G) : G);
            }
        };
        if (live == kTok) gather(std::true_type());
        else gather(std::false_type());
        f2 g;
        if (!enter_span<CL>(maps, k, warp, A, G, state, g, ok, a.err)) break;
        E *dx = static_cast<E *>(a.dx) + row, *dw = static_cast<E *>(a.dw) + row;
        float *dla = a.dla + row;
        auto sweep = [&](auto whole) {
#pragma unroll
            for (int t = kTok - 1; t >= 0; --t) {
                if (!decltype(whole)::value && t >= live) continue;
                const long long at = (long long)t * a.C;
                g = add2(get(2, dy, t), g);
                store_pair<EVEN>(dx + at, c, a.C, mul2(g, get(1, w, t)));
                store_pair<EVEN>(dw + at, c, a.C, mul2(g, get(0, x, t)));
                g = mul2(g, al[t]);
                store_pair<EVEN>(dla + at, c, a.C, mul2(g, hp[t]));
            }
        };
        if (live == kTok) sweep(std::true_type());
        else sweep(std::false_type());
        if (SRC == kTile) {
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(empty + st);
            if (threadIdx.x == 0 && sp >= S::COUNT) {
                if (sm100::mbar_wait(empty + st, ph, a.err))
                    fetch_span<E, 3>(dyn + st * S::BYTES, tm, full + st, c_cta, seq + first_token(sp - S::COUNT));
                else
                    ok = false;
            }
            if (++st == S::COUNT) st = 0, ph ^= 1;
        }
    }
    if (__builtin_expect(!ok, 0)) {
        if (SRC == kTile && threadIdx.x == 0) drain<S::COUNT>(full, st, ph, sp + 1, a.err);
        if (CL) sm100::leave_cluster();
        return;
    }
    if (a.dh0 && warp == 0 && pl.rank == 0) store_pair<EVEN>(a.dh0 + (long long)pl.b * a.C, c, a.C, state);
}

template <typename E>
__global__ void __launch_bounds__(256) scan_step_kernel(const ScanArgs a, float *h)
{
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= (long long)a.B * a.C) return;
    const float u = to_f32(static_cast<const E *>(a.x)[i]) * to_f32(static_cast<const E *>(a.w)[i]);
    const float v = fmaf(expf(a.la[i]), h[i], u);
    h[i] = v;
    static_cast<E *>(a.y)[i] = from_f32<E>(v);
}

// Four elements a thread.
template <typename E>
__global__ void __launch_bounds__(256) scan_step4_kernel(const ScanArgs a, float *h)
{
    const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= (long long)a.B * a.C) return;
    const float4 x = load4(static_cast<const E *>(a.x) + i), w = load4(static_cast<const E *>(a.w) + i), l = load4(a.la + i);
    float4 v = load4(h + i);
    v.x = fmaf(expf(l.x), v.x, x.x * w.x);
    v.y = fmaf(expf(l.y), v.y, x.y * w.y);
    v.z = fmaf(expf(l.z), v.z, x.z * w.z);
    v.w = fmaf(expf(l.w), v.w, x.w * w.w);
    store4(h + i, v);
    store4(static_cast<E *>(a.y) + i, v);
}

// CTAs of a cluster: as many as the device holds beside the channels' own CTAs, and no
// more than the sequence has spans.
int cluster_size(const ScanArgs &a, int num_sms)
{
    const long long tiles = (long long)((a.C + kChan - 1) / kChan) * a.B;
    int cs = 1;
    while (cs < kMaxCluster && tiles * cs * 2 <= 2LL * num_sms && (long long)cs * kSpan < a.T) cs *= 2;
    return cs;
}

template <auto kern>
cudaError_t launch(const ScanArgs &a, int cs, int smem, const SpanMaps &tm, cudaStream_t stream)
{
    static std::atomic<unsigned long long> set{0};
    cudaError_t e = ensure_smem_limit(kern, smem, set);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((a.C + kChan - 1) / kChan) * cs, a.B);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cs;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cs > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a, cs, tm);
}

// Tiles by TMA need rows of a multiple of 16 bytes and row numbers that fit its coordinates.
template <typename E>
Source source_of(const ScanArgs &a)
{
    if (a.C % (16 / sizeof(E)) == 0 && (long long)a.B * a.T + kSpan * kMaxCluster < 0x7fffffffLL) return kTile;
    return a.C % 2 == 0 ? kEven : kOdd;
}

template <typename E, Source SRC>
cudaError_t fwd_impl(const ScanArgs &a, int num_sms, cudaStream_t stream)
{
    const int cs = cluster_size(a, num_sms);
    SpanMaps tm{};
    int smem = 0;
    if (SRC == kTile) {
        const long long rows = (long long)a.B * a.T;
        const bool bf16 = sizeof(E) == 2;
        smem = Stage<E, 2>::BYTES * Stage<E, 2>::COUNT;
        if (!make_plane_map(&tm.la, a.la, false, a.C, rows, kChan, kSpan) || !make_plane_map(&tm.e[0], a.x, bf16, a.C, rows, kChan, kSpan) ||
            !make_plane_map(&tm.e[1], a.w, bf16, a.C, rows, kChan, kSpan))
            return cudaErrorInvalidValue;
    }
    return cs > 1 ? launch<scan_fwd_kernel<E, SRC, true>>(a, cs, smem, tm, stream)
                  : launch<scan_fwd_kernel<E, SRC, false>>(a, 1, smem, tm, stream);
}
template <typename E, Source SRC>
cudaError_t bwd_impl(const ScanArgs &a, int num_sms, cudaStream_t stream)
{
    const int cs = cluster_size(a, num_sms);
    SpanMaps tm{};
    int smem = 0;
    if (SRC == kTile) {
        const long long rows = (long long)a.B * a.T;
        const bool bf16 = sizeof(E) == 2;
        smem = Stage<E, 3>::BYTES * Stage<E, 3>::COUNT;
        if (!make_plane_map(&tm.la, a.la, false, a.C, rows, kChan, kSpan) || !make_plane_map(&tm.e[0], a.x, bf16, a.C, rows, kChan, kSpan) ||
            !make_plane_map(&tm.e[1], a.w, bf16, a.C, rows, kChan, kSpan) || !make_plane_map(&tm.e[2], a.dy, bf16, a.C, rows, kChan, kSpan))
            return cudaErrorInvalidValue;
    }
    return cs > 1 ? launch<scan_bwd_kernel<E, SRC, true>>(a, cs, smem, tm, stream)
                  : launch<scan_bwd_kernel<E, SRC, false>>(a, 1, smem, tm, stream);
}

template <typename E>
cudaError_t fwd_by_source(const ScanArgs &a, int num_sms, cudaStream_t stream)
{
    switch (source_of<E>(a)) {
    case kTile: return fwd_impl<E, kTile>(a, num_sms, stream);
    case kEven: return fwd_impl<E, kEven>(a, num_sms, stream);
    default: return fwd_impl<E, kOdd>(a, num_sms, stream);
    }
}
template <typename E>
cudaError_t bwd_by_source(const ScanArgs &a, int num_sms, cudaStream_t stream)
{
    switch (source_of<E>(a)) {
    case kTile: return bwd_impl<E, kTile>(a, num_sms, stream);
    case kEven: return bwd_impl<E, kEven>(a, num_sms, stream);
    default: return bwd_impl<E, kOdd>(a, num_sms, stream);
    }
}

}  // namespace

cudaError_t launch_scan_fwd(const ScanArgs &a, bool bf16, int num_sms, cudaStream_t stream)
{
    return bf16 ? fwd_by_source<__nv_bfloat16>(a, num_sms, stream) : fwd_by_source<float>(a, num_sms, stream);
}

cudaError_t launch_scan_bwd(const ScanArgs &a, bool bf16, int num_sms, cudaStream_t stream)
{
    return bf16 ? bwd_by_source<__nv_bfloat16>(a, num_sms, stream) : bwd_by_source<float>(a, num_sms, stream);
}

cudaError_t launch_scan_step(const ScanArgs &a, float *h, bool bf16, cudaStream_t stream)
{
    const long long n = (long long)a.B * a.C, per = n % 4 == 0 ? 1024 : 256, blocks = (n + per - 1) / per;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks), block(256);
    if (n % 4 == 0)
        return bf16 ? launch_plain(scan_step4_kernel<__nv_bfloat16>, grid, block, 0, stream, a, h)
                    : launch_plain(scan_step4_kernel<float>, grid, block, 0, stream, a, h);
    return bf16 ? launch_plain(scan_step_kernel<__nv_bfloat16>, grid, block, 0, stream, a, h)
                : launch_plain(scan_step_kernel<float>, grid, block, 0, stream, a, h);
}

}  // namespace gdn2
