// scan.cu -- the gated linear recurrence h_t = alpha_t h_{t-1} + w_t x_t per
// channel: forward, backward and single step.
//
// One pass over the data.  A CTA takes 64 channels and 128 tokens at a time: its eight
// warps hold 16 tokens each in registers (two channels a lane), reduce them to the map
// h -> A h + H of their span, and compose the maps of the spans before theirs through
// shared memory; then every warp knows the state it starts from and runs its tokens.
// When channels alone do not fill the device, a cluster of up to eight CTAs takes
// consecutive spans of 128 tokens of the same channels and exchanges its maps through
// distributed shared memory.  The walk over the sequence carries the state in registers.
// Bound by HBM.
//
// Backward: the same with time reversed, on c_t = alpha_t g_t (the gradient that leaves a
// token towards the past): c -> A c + G.  h_{t-1} comes from the forward's checkpoints,
// one per 16 tokens, recomputed in fp32.
#include <cooperative_groups.h>

#include "common.cuh"
#include "hybrid.h"
#include "packed.cuh"

namespace gdn2 {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kTok = kScanBlock;          // tokens of a warp
constexpr int kSpan = kWarps * kTok;      // tokens of a CTA
constexpr int kChan = 64;                 // channels of a CTA
constexpr int kMaxCluster = 8;

// The pair of channels c, c + 1 of a row; 0 (or `fill`) outside [0, C).
template <bool EVEN, typename E>
__device__ __forceinline__ f2 load_pair(const E *row, int c, int C, float fill = 0.f)
{
    if constexpr (EVEN) {
        if (c >= C) return both(fill);
        alignas(8) E e[2];
        if constexpr (sizeof(E) == 4) *reinterpret_cast<float2 *>(e) = __ldg(reinterpret_cast<const float2 *>(row + c));
        else *reinterpret_cast<uint32_t *>(e) = __ldg(reinterpret_cast<const uint32_t *>(row + c));
        return pair_of(e);
    } else {
        return pack2(c < C ? to_f32(row[c]) : fill, c + 1 < C ? to_f32(row[c + 1]) : fill);
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
};
// From this warp's map and the running state: the state entering its span; `state`
// becomes the one behind the whole cluster's span.  `order` is the warp's (or the CTA's)
// position along the walk.
template <bool CL>
__device__ __forceinline__ f2 enter_span(Maps &m, int parity, int order, f2 A, f2 H, f2 &state)
{
    const int lane = threadIdx.x & 31;
    m.warp[parity][order][lane] = make_ulonglong2(A, H);
    __syncthreads();
    f2 pa = both(1.f), ph = 0, ta = both(1.f), th = 0;  // before this warp, and in all
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w == order) pa = ta, ph = th;
        const ulonglong2 v = m.warp[parity][w][lane];
        ta = mul2(v.x, ta);
        th = fma2(v.x, th, v.y);
    }
    f2 in = state;
    if constexpr (CL) {
        cg::cluster_group cluster = cg::this_cluster();
        const int size = cluster.num_blocks(), rank = cluster.block_rank();
        if (order < size) *cluster.map_shared_rank(&m.cta[parity][rank][lane], order) = make_ulonglong2(ta, th);
        cluster.sync();
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
    return fma2(pa, in, ph);
}

// Where a CTA works: channels, batch, and its place among the CTAs of its span.
struct Place {
    int c, b, rank, size;
    __device__ __forceinline__ Place(int csize)
        : c((int)(blockIdx.x / csize) * kChan + 2 * (threadIdx.x & 31)), b(blockIdx.y), rank(blockIdx.x % csize), size(csize) {}
};

template <typename E, bool EVEN, bool CL>
__global__ void __launch_bounds__(kThreads, 2) scan_fwd_kernel(const ScanArgs a, int csize)
{
    __shared__ Maps maps;
    const Place pl(csize);
    const int warp = threadIdx.x >> 5, c = pl.c;
    const long long seq = (long long)pl.b * a.T;
    const int nblk = (a.T + kTok - 1) / kTok;
    f2 state = a.h0 ? load_pair<EVEN>(a.h0 + (long long)pl.b * a.C, c, a.C) : 0;
    if constexpr (CL) cg::this_cluster().sync();  // every CTA has started (and read h0, which h_T may alias)
    int parity = 0;
    for (long long s0 = 0; s0 < a.T; s0 += (long long)kSpan * pl.size, parity ^= 1) {
        const long long t0 = s0 + pl.rank * kSpan + warp * kTok;
        const int live = t0 >= a.T ? 0 : a.T - t0 < kTok ? (int)(a.T - t0) : kTok;
        const long long row = (seq + t0) * a.C;
        f2 al[kTok], u[kTok];
#pragma unroll
        for (int t = 0; t < kTok; ++t) {
            const long long at = row + (long long)t * a.C;
            const bool on = t < live;
            al[t] = on ? load_pair<EVEN>(a.la + at, c, a.C) : 0;
            u[t] = on ? mul2(load_pair<EVEN>(static_cast<const E *>(a.x) + at, c, a.C),
                             load_pair<EVEN>(static_cast<const E *>(a.w) + at, c, a.C)) : 0;
        }
        f2 A = both(1.f), H = 0;
#pragma unroll
        for (int t = 0; t < kTok; ++t) {
            al[t] = exp_pair(al[t]);
            A = mul2(al[t], A);
            H = fma2(al[t], H, u[t]);
        }
        f2 h = enter_span<CL>(maps, parity, warp, A, H, state);
        if (live > 0) {
            if (a.ckpt) store_pair<EVEN>(a.ckpt + ((long long)pl.b * nblk + t0 / kTok) * a.C, c, a.C, h);
#pragma unroll
            for (int t = 0; t < kTok; ++t) {
                h = fma2(al[t], h, u[t]);
                if (t < live) store_pair<EVEN>(static_cast<E *>(a.y) + row + (long long)t * a.C, c, a.C, h);
            }
        }
    }
    if (a.h_T && warp == 0 && pl.rank == 0) store_pair<EVEN>(a.h_T + (long long)pl.b * a.C, c, a.C, state);
}

template <typename E, bool EVEN, bool CL>
__global__ void __launch_bounds__(kThreads, 2) scan_bwd_kernel(const ScanArgs a, int csize)
{
    __shared__ Maps maps;
    const Place pl(csize);
    const int warp = threadIdx.x >> 5, c = pl.c;
    const long long seq = (long long)pl.b * a.T;
    const int nblk = (a.T + kTok - 1) / kTok;
    f2 state = a.dh_T ? load_pair<EVEN>(a.dh_T + (long long)pl.b * a.C, c, a.C) : 0;
    if constexpr (CL) cg::this_cluster().sync();  // every CTA has started (and read dh_T, which dh0 may alias)
    int parity = 0;
    const long long step = (long long)kSpan * pl.size, spans = (a.T + step - 1) / step;
    for (long long sp = spans - 1; sp >= 0; --sp, parity ^= 1) {
        // along the walk the last tokens come first: rank 0 and warp 0 take the latest
        const long long t0 = sp * step + (pl.size - 1 - pl.rank) * kSpan + (kWarps - 1 - warp) * kTok;
        const int live = t0 >= a.T ? 0 : a.T - t0 < kTok ? (int)(a.T - t0) : kTok;
        const long long row = (seq + t0) * a.C;
        const E *x = static_cast<const E *>(a.x) + row, *w = static_cast<const E *>(a.w) + row;
        f2 al[kTok], hp[kTok], dy[kTok];
#pragma unroll
        for (int t = 0; t < kTok; ++t) {
            const long long at = (long long)t * a.C;
            const bool on = t < live;
            al[t] = on ? load_pair<EVEN>(a.la + row + at, c, a.C) : 0;
            dy[t] = on ? load_pair<EVEN>(static_cast<const E *>(a.dy) + row + at, c, a.C) : 0;
            hp[t] = on ? mul2(load_pair<EVEN>(x + at, c, a.C), load_pair<EVEN>(w + at, c, a.C)) : 0;
        }
        f2 h = live ? load_pair<EVEN>(a.ckpt + ((long long)pl.b * nblk + t0 / kTok) * a.C, c, a.C) : 0;
#pragma unroll
        for (int t = 0; t < kTok; ++t) {
            al[t] = exp_pair(al[t]);
            const f2 next = fma2(al[t], h, hp[t]);
            hp[t] = h;
            h = next;
        }
        f2 A = both(1.f), G = 0;
#pragma unroll
        for (int t = kTok - 1; t >= 0; --t) {
            A = mul2(al[t], A);
            G = mul2(al[t], add2(dy[t], G));
        }
        f2 g = enter_span<CL>(maps, parity, warp, A, G, state);
#pragma unroll
        for (int t = kTok - 1; t >= 0; --t) {
            if (t >= live) continue;
            const long long at = (long long)t * a.C;
            g = add2(dy[t], g);
            // (x and w again, from cache: kept in registers they would halve the CTAs of an SM)
            store_pair<EVEN>(static_cast<E *>(a.dx) + row + at, c, a.C, mul2(g, load_pair<EVEN>(w + at, c, a.C)));
            store_pair<EVEN>(static_cast<E *>(a.dw) + row + at, c, a.C, mul2(g, load_pair<EVEN>(x + at, c, a.C)));
            g = mul2(g, al[t]);
            store_pair<EVEN>(a.dla + row + at, c, a.C, mul2(g, hp[t]));
        }
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
cudaError_t launch(const ScanArgs &a, int cs, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((a.C + kChan - 1) / kChan) * cs, a.B);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cs;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cs > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a, cs);
}

template <typename E, bool EVEN>
cudaError_t fwd_impl(const ScanArgs &a, int num_sms, cudaStream_t stream)
{
    const int cs = cluster_size(a, num_sms);
    return cs > 1 ? launch<scan_fwd_kernel<E, EVEN, true>>(a, cs, stream) : launch<scan_fwd_kernel<E, EVEN, false>>(a, 1, stream);
}
template <typename E, bool EVEN>
cudaError_t bwd_impl(const ScanArgs &a, int num_sms, cudaStream_t stream)
{
    const int cs = cluster_size(a, num_sms);
    return cs > 1 ? launch<scan_bwd_kernel<E, EVEN, true>>(a, cs, stream) : launch<scan_bwd_kernel<E, EVEN, false>>(a, 1, stream);
}

}  // namespace

cudaError_t launch_scan_fwd(const ScanArgs &a, bool bf16, int num_sms, cudaStream_t stream)
{
    if (a.C % 2 == 0) return bf16 ? fwd_impl<__nv_bfloat16, true>(a, num_sms, stream) : fwd_impl<float, true>(a, num_sms, stream);
    return bf16 ? fwd_impl<__nv_bfloat16, false>(a, num_sms, stream) : fwd_impl<float, false>(a, num_sms, stream);
}

cudaError_t launch_scan_bwd(const ScanArgs &a, bool bf16, int num_sms, cudaStream_t stream)
{
    if (a.C % 2 == 0) return bf16 ? bwd_impl<__nv_bfloat16, true>(a, num_sms, stream) : bwd_impl<float, true>(a, num_sms, stream);
    return bf16 ? bwd_impl<__nv_bfloat16, false>(a, num_sms, stream) : bwd_impl<float, false>(a, num_sms, stream);
}

cudaError_t launch_scan_step(const ScanArgs &a, float *h, bool bf16, cudaStream_t stream)
{
    const long long n = (long long)a.B * a.C, per = n % 4 == 0 ? 1024 : 256, blocks = (n + per - 1) / per;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)blocks;
    if (n % 4 == 0) {
        if (bf16) scan_step4_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a, h);
        else scan_step4_kernel<float><<<grid, 256, 0, stream>>>(a, h);
    } else {
        if (bf16) scan_step_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a, h);
        else scan_step_kernel<float><<<grid, 256, 0, stream>>>(a, h);
    }
    return cudaGetLastError();
}

}  // namespace gdn2
