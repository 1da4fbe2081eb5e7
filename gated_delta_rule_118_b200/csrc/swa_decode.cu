// swa_decode.cu -- one token of the windowed attention against a ring cache.
//
// A cluster of CTAs shares one (batch, key/value head): each CTA takes a run of
// the visible positions, each of its warps every fourth group of them, and the
// partial (max, sum, output) triples are joined through shared memory, then
// through distributed shared memory -- one launch, no workspace.
#include <cooperative_groups.h>

#include "launch.h"
#include "swa_common.cuh"

namespace gdn2 {
namespace {

using namespace swa;
namespace cg = cooperative_groups;

constexpr int kWarps = 4;

// Visible positions in order (sinks behind the window, then the window) -> cache slots.
struct Visible {
    int ns, lo, n, sinks, ring, first, base;
    __device__ __forceinline__ Visible(int P, int window, int sinks_, int slots)
    {
        sinks = sinks_;
        ring = slots - sinks;
        lo = P - window + 1 > 0 ? P - window + 1 : 0;
        ns = sinks < lo ? sinks : lo;
        n = ns + P + 1 - lo;
        first = lo > sinks ? lo : sinks;  // first position of the window that lives in the ring
        base = (first - sinks) % ring;
    }
    __device__ __forceinline__ int position(int t) const { return t < ns ? t : lo + t - ns; }
    __device__ __forceinline__ int slot(int p) const
    {
        if (p < sinks) return p;
        const int r = base + p - first;  // below 2 * ring: a window spans at most the ring
        return sinks + (r >= ring ? r - ring : r);
    }
};

template <typename E>
__device__ __forceinline__ void put_new_token(const SwaDecodeArgs &a, int b, int hk, int P, const E *kn, const E *vn)
{
    const int s = P < a.sinks ? P : a.sinks + (P - a.sinks) % (a.slots - a.sinks);
    const long long at = (((long long)b * a.slots + s) * a.Hk + hk) * a.d;
    for (int c = threadIdx.x * 4; c < a.d; c += blockDim.x * 4) {
        store4(static_cast<E *>(a.kc) + at + c, load4(kn + c));
        store4(static_cast<E *>(a.vc) + at + c, load4(vn + c));
    }
}

// GC query heads of the group per CTA; lanes hold 4 channels each of D / 4 lanes per key.
template <typename E, int D, int GC>
__global__ void __launch_bounds__(kWarps * 32) decode_kernel(const SwaDecodeArgs a, int nsplit, int nchunk)
{
    constexpr int LPR = D / 4, KPW = 32 / LPR;  // lanes per key, keys per warp step
    constexpr int U = 4;                        // steps in flight
    __shared__ float sm_m[kWarps][GC], sm_l[kWarps][GC], sm_o[kWarps][GC][D];
    __shared__ float cm[GC], cl[GC], co[GC][D];
    const int split = blockIdx.x, hk = blockIdx.y / nchunk, chunk = blockIdx.y % nchunk, b = blockIdx.z;
    const int G = a.Hq / a.Hk, g0 = chunk * GC, ng = min(GC, G - g0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / LPR, x = lane % LPR * 4;
    E *out = static_cast<E *>(a.o) + ((long long)b * a.Hq + hk * G + g0) * D;
    const int P = a.pos[b];
    if (P < 0) {  // no sequence in this row
        if (split == 0)
            for (int c = threadIdx.x; c < ng * D; c += blockDim.x) out[c] = from_f32<E>(0.f);
        return;
    }
    const E *kn = static_cast<const E *>(a.k) + b * a.ks[0] + hk * a.ks[1];
    const E *vn = static_cast<const E *>(a.v) + b * a.vs[0] + hk * a.vs[1];
    if (split == 0 && chunk == 0) put_new_token<E>(a, b, hk, P, kn, vn);
    const Visible vis(P, a.window, a.sinks, a.slots);
    const long long cache0 = ((long long)b * a.slots * a.Hk + hk) * D, cstep = (long long)a.Hk * D;
    const E *kc = static_cast<const E *>(a.kc) + cache0, *vc = static_cast<const E *>(a.vc) + cache0;

    float q[GC][4], m[GC], l[GC], o[GC][4];
#pragma unroll
    for (int g = 0; g < GC; ++g) {
        const E *qr = static_cast<const E *>(a.q) + b * a.qs[0] + (long long)(hk * G + g0 + min(g, ng - 1)) * a.qs[1];
        const float4 f = load4(qr + x);
        const float sc = a.scale * kLog2E;
        q[g][0] = f.x * sc; q[g][1] = f.y * sc; q[g][2] = f.z * sc; q[g][3] = f.w * sc;
        m[g] = -INFINITY;
        l[g] = o[g][0] = o[g][1] = o[g][2] = o[g][3] = 0.f;
    }
    const int per = (vis.n + nsplit - 1) / nsplit;
    const int t0 = split * per, t1 = min(vis.n, t0 + per);
    for (int t = t0 + warp * KPW * U; t < t1; t += kWarps * KPW * U) {
        float4 kf[U], vf[U];
        bool on[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int tt = t + u * KPW + sub;
            on[u] = tt < t1;
            const int p = vis.position(on[u] ? tt : t0);
            const long long at = vis.slot(p) * cstep;
            kf[u] = load4((p == P ? kn : kc + at) + x);
            vf[u] = load4((p == P ? vn : vc + at) + x);
        }
#pragma unroll
        for (int g = 0; g < GC; ++g) {
            float s[U], mx = m[g];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                s[u] = fmaf(q[g][0], kf[u].x, fmaf(q[g][1], kf[u].y, fmaf(q[g][2], kf[u].z, q[g][3] * kf[u].w)));
#pragma unroll
                for (int w = LPR / 2; w; w >>= 1) s[u] += __shfl_xor_sync(~0u, s[u], w);
                s[u] = on[u] ? s[u] : -INFINITY;
                mx = fmaxf(mx, s[u]);
            }
            const float ms = mx == -INFINITY ? 0.f : mx, f = exp2f(m[g] - ms);
            m[g] = mx;
            l[g] *= f;
#pragma unroll
            for (int c = 0; c < 4; ++c) o[g][c] *= f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!on[u]) continue;
                const float e = exp2f(s[u] - ms);
                l[g] += e;
                o[g][0] = fmaf(e, vf[u].x, o[g][0]);
                o[g][1] = fmaf(e, vf[u].y, o[g][1]);
                o[g][2] = fmaf(e, vf[u].z, o[g][2]);
                o[g][3] = fmaf(e, vf[u].w, o[g][3]);
            }
        }
    }
    // the keys of a warp's sub-rows, then the warps, then the CTAs of the cluster
#pragma unroll
    for (int g = 0; g < GC; ++g) {
#pragma unroll
        for (int w = LPR; w < 32; w <<= 1) {
            const float mo = __shfl_xor_sync(~0u, m[g], w), mn = fmaxf(m[g], mo), ms = mn == -INFINITY ? 0.f : mn;
            const float f = exp2f(m[g] - ms), fo = exp2f(mo - ms);
            l[g] = l[g] * f + __shfl_xor_sync(~0u, l[g], w) * fo;
#pragma unroll
            for (int c = 0; c < 4; ++c) o[g][c] = o[g][c] * f + __shfl_xor_sync(~0u, o[g][c], w) * fo;
            m[g] = mn;
        }
        if (lane < LPR) {
#pragma unroll
            for (int c = 0; c < 4; ++c) sm_o[warp][g][x + c] = o[g][c];
            if (lane == 0) sm_m[warp][g] = m[g], sm_l[warp][g] = l[g];
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < GC * D; c += blockDim.x) {
        const int g = c / D, d = c % D;
        float mn = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mn = fmaxf(mn, sm_m[w][g]);
        const float ms = mn == -INFINITY ? 0.f : mn;
        float sl = 0.f, so = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2f(sm_m[w][g] - ms);
            sl = fmaf(sm_l[w][g], f, sl);
            so = fmaf(sm_o[w][g][d], f, so);
        }
        co[g][d] = so;
        if (d == 0) cm[g] = mn, cl[g] = sl;
    }
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    if (split < ng) {  // heads dealt to the CTAs of the cluster
        for (int g = split; g < ng; g += nsplit)
            for (int d = threadIdx.x; d < D; d += blockDim.x) {
                float mn = -INFINITY;
                for (int r = 0; r < nsplit; ++r) mn = fmaxf(mn, *cluster.map_shared_rank(&cm[g], r));
                const float ms = mn == -INFINITY ? 0.f : mn;
                float sl = 0.f, so = 0.f;
                for (int r = 0; r < nsplit; ++r) {
                    const float f = exp2f(*cluster.map_shared_rank(&cm[g], r) - ms);
                    sl = fmaf(*cluster.map_shared_rank(&cl[g], r), f, sl);
                    so = fmaf(*cluster.map_shared_rank(&co[g][d], r), f, so);
                }
                out[g * D + d] = from_f32<E>(sl == 0.f ? 0.f : so / sl);
            }
    }
    cluster.sync();
}

template <typename E, int D, int GC>
cudaError_t impl(const SwaDecodeArgs &a, int num_sms, cudaStream_t stream)
{
    const int G = a.Hq / a.Hk, nchunk = (G + GC - 1) / GC;
    if ((long long)a.Hk * nchunk > 65535) return cudaErrorInvalidValue;
    const long long ctas = (long long)a.B * a.Hk * nchunk;
    int nsplit = 1;
    while (nsplit < 8 && ctas * nsplit < 2LL * num_sms && (a.window + a.sinks) / (nsplit * 2) >= 64) nsplit *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(nsplit, a.Hk * nchunk, a.B);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = nsplit;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, decode_kernel<E, D, GC>, a, nsplit, nchunk);
}

template <typename E, int D>
cudaError_t by_group(const SwaDecodeArgs &a, int num_sms, cudaStream_t stream)
{
    const int G = a.Hq / a.Hk;
    if (G == 1) return impl<E, D, 1>(a, num_sms, stream);
    if (G == 2) return impl<E, D, 2>(a, num_sms, stream);
    return impl<E, D, 4>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_swa_decode(const SwaDecodeArgs &a, bool bf16, int num_sms, cudaStream_t stream)
{
    if (bf16)
        return a.d == 128 ? by_group<__nv_bfloat16, 128>(a, num_sms, stream)
                          : by_group<__nv_bfloat16, 64>(a, num_sms, stream);
    return a.d == 128 ? by_group<float, 128>(a, num_sms, stream) : by_group<float, 64>(a, num_sms, stream);
}

}  // namespace gdn2
