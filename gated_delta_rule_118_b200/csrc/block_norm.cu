// block_norm.cu -- the norms around a block, fused with its gate and residual
// scale, forward and backward.
//
// A row stays in registers: 8 columns a thread, up to 512 threads a CTA, and rows of
// more than 4096 columns across a cluster of up to four CTAs that exchange their sums
// through distributed shared memory.  So every tensor is read and written once.  CTAs
// walk over rows with the grid's stride: the vectors (weights, scales) and the backward's
// column sums stay in registers, and bf16 rows are fetched one row ahead, since the row
// sums of one row (two in the forward, three in the backward) would otherwise leave the
// memory idle.  Bound by HBM.
//
// The backward's sums over rows (for the three vectors' gradients) are added in a fixed
// order: each CTA over its rows, then a small kernel over the CTAs.  dw_post and
// dres_scale are the same sum times the other vector, so two sums are kept, not three.
#include <cooperative_groups.h>

#include "common.cuh"
#include "hybrid.h"
#include "launch.h"
#include "sm100.cuh"

namespace gdn2 {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxThreads = 512;
constexpr int kMaxCols = 8 * kMaxThreads;  // columns of one CTA

// Eight elements of a row: contiguous ones (16-byte loads), or one every NT columns for
// rows that are not a multiple of 8 long.
template <typename E, bool VEC>
struct Eight {
    E e[8];
    __device__ __forceinline__ void load(const E *row, int c0, int tid, int nt, int cols)
    {
        if constexpr (VEC) {
            const bool on = c0 + tid * 8 < cols;
            constexpr int W = sizeof(E) / 2;  // 16-byte words
#pragma unroll
            for (int w = 0; w < W; ++w)
                reinterpret_cast<uint4 *>(e)[w] =
                    on ? __ldcs(reinterpret_cast<const uint4 *>(row + c0 + tid * 8) + w) : make_uint4(0, 0, 0, 0);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = c0 + tid + i * nt;
                e[i] = c < cols ? row[c] : from_f32<E>(0.f);
            }
        }
    }
    __device__ __forceinline__ float operator[](int i) const { return to_f32(e[i]); }
};
template <typename E, bool VEC>
__device__ __forceinline__ void store_eight(E *row, const float (&f)[8], int c0, int tid, int nt, int cols)
{
    if constexpr (VEC) {
        if (c0 + tid * 8 < cols) {
            store4(row + c0 + tid * 8, make_float4(f[0], f[1], f[2], f[3]));
            store4(row + c0 + tid * 8 + 4, make_float4(f[4], f[5], f[6], f[7]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c0 + tid + i * nt < cols) row[c0 + tid + i * nt] = from_f32<E>(f[i]);
    }
}
template <bool VEC>
__device__ __forceinline__ int column(int c0, int tid, int nt, int i)
{
    return VEC ? c0 + tid * 8 + i : c0 + tid + i * nt;
}

// 1 / (1 + 2^(-x log2 e)): both steps are accurate to about 2^-22, which the sums over
// rows need (a half-precision hyperbolic tangent would show in their gradients).
__device__ __forceinline__ float sigmoid(float x)
{
    float t, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(-1.4426950408889634f * x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + t));
    return r;
}

// Sums of N values over the CTA, and over the cluster with CL, left in every thread.
// Slots alternate, so the next sum may start while slower threads still read this one.
template <bool CL>
struct RowSums {
    float (*warp_part)[2][kMaxThreads / 32];  // [slot][value][warp]
    float (*cta_part)[2][4];                  // [slot][value][CTA of the cluster]
    int slot = 0;
    template <int N>
    __device__ __forceinline__ void operator()(float (&v)[N])
    {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = (blockDim.x + 31) >> 5;
#pragma unroll
        for (int n = 0; n < N; ++n) {
#pragma unroll
            for (int o = 16; o; o >>= 1) v[n] += __shfl_xor_sync(~0u, v[n], o);
            if (lane == 0) warp_part[slot][n][warp] = v[n];
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            v[n] = 0.f;
            for (int w = 0; w < nw; ++w) v[n] += warp_part[slot][n][w];
        }
        if constexpr (CL) {
            cg::cluster_group cluster = cg::this_cluster();
            const int size = cluster.num_blocks(), rank = cluster.block_rank();
            if (threadIdx.x < size)
#pragma unroll
                for (int n = 0; n < N; ++n) *cluster.map_shared_rank(&cta_part[slot][n][rank], threadIdx.x) = v[n];
            cluster.sync();
#pragma unroll
            for (int n = 0; n < N; ++n) {
                v[n] = 0.f;
                for (int c = 0; c < size; ++c) v[n] += cta_part[slot][n][c];
            }
        }
        slot ^= 1;
    }
};

template <typename E, bool VEC, bool CL>
__global__ void __launch_bounds__(kMaxThreads) norm_fwd_kernel(const NormArgs a, int cols_per_cta, int csize)
{
    __shared__ float warp_part[2][2][kMaxThreads / 32], cta_part[2][2][4];
    RowSums<CL> sums{warp_part, cta_part};
    const int tid = threadIdx.x, nt = blockDim.x;
    const int c0 = CL ? (int)(blockIdx.x % csize) * cols_per_cta : 0, cols = min(a.D, c0 + cols_per_cta);
    const long long first = blockIdx.x / csize, step = gridDim.x / csize;
    const float rd = 1.f / a.D;
    float t[8], wq[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = column<VEC>(c0, tid, nt, i);
        const bool on = c < cols;
        t[i] = on ? a.res[c] * a.w_post[c] : 0.f;
        wq[i] = on ? a.w_pre[c] : 0.f;
    }
    auto in = [&](const void *p, long long n) { return static_cast<const E *>(p) + n * a.D; };
    constexpr bool AHEAD = sizeof(E) == 2;
    Eight<E, VEC> y, r, g;
    auto fetch = [&](long long n) {
        y.load(in(a.y, n), c0, tid, nt, cols);
        r.load(in(a.r, n), c0, tid, nt, cols);
        if (a.g) g.load(in(a.g, n), c0, tid, nt, cols);
    };
    if (AHEAD && first < a.N) fetch(first);
    for (long long n = first; n < a.N; n += step) {
        if (!AHEAD) fetch(n);
        float yv[8], r1[8], gt[8], s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            yv[i] = y[i];
            r1[i] = r[i];
            gt[i] = a.g ? sigmoid(g[i]) * t[i] : t[i];
            s[0] = fmaf(yv[i], yv[i], s[0]);
        }
        if (AHEAD && n + step < a.N) fetch(n + step);
        sums(s);
        const float iy = rsqrtf(fmaf(s[0], rd, a.eps));
        s[0] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            r1[i] = fmaf(gt[i], yv[i] * iy, r1[i]);
            s[0] = fmaf(r1[i], r1[i], s[0]);
        }
        store_eight<E, VEC>(static_cast<E *>(a.r_out) + n * a.D, r1, c0, tid, nt, cols);
        sums(s);
        const float ir = rsqrtf(fmaf(s[0], rd, a.eps));
#pragma unroll
        for (int i = 0; i < 8; ++i) r1[i] *= ir * wq[i];
        store_eight<E, VEC>(static_cast<E *>(a.x_out) + n * a.D, r1, c0, tid, nt, cols);
    }
    if constexpr (CL) cg::this_cluster().sync();  // no CTA leaves while another may still write its slots
}

template <typename E, bool VEC, bool CL>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_kernel(const NormArgs a, int cols_per_cta, int csize)
{
    __shared__ float warp_part[2][2][kMaxThreads / 32], cta_part[2][2][4];
    RowSums<CL> sums{warp_part, cta_part};
    const int tid = threadIdx.x, nt = blockDim.x;
    const int c0 = CL ? (int)(blockIdx.x % csize) * cols_per_cta : 0, cols = min(a.D, c0 + cols_per_cta);
    const long long first = blockIdx.x / csize, step = gridDim.x / csize;
    const float rd = 1.f / a.D;
    float t[8], wq[8], bsum[8] = {}, psum[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = column<VEC>(c0, tid, nt, i);
        const bool on = c < cols;
        t[i] = on ? a.res[c] * a.w_post[c] : 0.f;
        wq[i] = on ? a.w_pre[c] : 0.f;
    }
    auto in = [&](const void *p, long long n) { return static_cast<const E *>(p) + n * a.D; };
    constexpr bool AHEAD = sizeof(E) == 2;
    Eight<E, VEC> y, r, g, dx, dr;
    auto fetch = [&](long long n) {
        y.load(in(a.y, n), c0, tid, nt, cols);
        r.load(in(a.r, n), c0, tid, nt, cols);
        if (a.g) g.load(in(a.g, n), c0, tid, nt, cols);
        dx.load(in(a.dx_out, n), c0, tid, nt, cols);
        dr.load(in(a.dr_out, n), c0, tid, nt, cols);
    };
    if (AHEAD && first < a.N) fetch(first);
    for (long long n = first; n < a.N; n += step) {
        if (!AHEAD) fetch(n);
        float yv[8], r1[8], gt[8], xv[8], dv[8], s[1] = {0.f}, s2[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            yv[i] = y[i];
            r1[i] = r[i];
            gt[i] = a.g ? sigmoid(g[i]) : 1.f;
            xv[i] = dx[i];
            dv[i] = dr[i];
            s[0] = fmaf(yv[i], yv[i], s[0]);
        }
        if (AHEAD && n + step < a.N) fetch(n + step);
        sums(s);
        const float iy = rsqrtf(fmaf(s[0], rd, a.eps));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            yv[i] *= iy;
            r1[i] = fmaf(t[i] * gt[i], yv[i], r1[i]);
            s2[0] = fmaf(r1[i], r1[i], s2[0]);
            s2[1] = fmaf(xv[i] * wq[i], r1[i], s2[1]);
        }
        sums(s2);
        const float ir = rsqrtf(fmaf(s2[0], rd, a.eps)), mx = s2[1] * rd * ir * ir;
        s[0] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            dv[i] = fmaf(ir, fmaf(xv[i], wq[i], -r1[i] * mx), dv[i]);
            psum[i] = fmaf(xv[i], r1[i] * ir, psum[i]);
            xv[i] = dv[i] * gt[i];            // gradient of the gated term, before its scale
            s[0] = fmaf(xv[i] * t[i], yv[i], s[0]);
        }
        store_eight<E, VEC>(static_cast<E *>(a.dr) + n * a.D, dv, c0, tid, nt, cols);
        sums(s);
        const float my = s[0] * rd;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float b = xv[i] * yv[i];
            bsum[i] += b;
            r1[i] = iy * fmaf(xv[i], t[i], -yv[i] * my);
            dv[i] = b * t[i] * (1.f - gt[i]);
        }
        store_eight<E, VEC>(static_cast<E *>(a.dy) + n * a.D, r1, c0, tid, nt, cols);
        if (a.g) store_eight<E, VEC>(static_cast<E *>(a.dg) + n * a.D, dv, c0, tid, nt, cols);
    }
    float *part = a.partial + first * 2 * a.D;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = column<VEC>(c0, tid, nt, i);
        if (c < cols) {
            part[c] = bsum[i];
            part[a.D + c] = psum[i];
        }
    }
    if constexpr (CL) cg::this_cluster().sync();
}

// 32 columns a CTA, its 8 warps over the partial rows.
__global__ void __launch_bounds__(256) norm_reduce_kernel(const NormArgs a, int rows)
{
    __shared__ float red[2][8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float b = 0.f, p = 0.f;
    if (c < a.D)
        for (int r = warp; r < rows; r += 8) {
            b += a.partial[(long long)r * 2 * a.D + c];
            p += a.partial[(long long)r * 2 * a.D + a.D + c];
        }
    red[0][warp][lane] = b;
    red[1][warp][lane] = p;
    __syncthreads();
    if (warp == 0 && c < a.D) {
        b = p = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            b += red[0][w][lane];
            p += red[1][w][lane];
        }
        a.dw_post[c] = b * a.res[c];
        a.dres[c] = b * a.w_post[c];
        a.dw_pre[c] = p;
    }
}

// CTAs of the cluster, columns and threads of each, and rows in flight.
struct NormPlan {
    int csize, cols, threads, rows;
};
NormPlan plan_norm(long long N, int D, int num_sms, int threads_per_sm)
{
    NormPlan p;
    p.csize = D <= kMaxCols ? 1 : D <= 2 * kMaxCols ? 2 : 4;
    p.cols = (D + p.csize - 1) / p.csize;
    p.cols = (p.cols + 7) / 8 * 8;
    p.threads = (p.cols + 255) / 256 * 32;
    const long long fit = (long long)num_sms * (threads_per_sm / p.threads > 32 ? 32 : threads_per_sm / p.threads) / p.csize;
    p.rows = (int)(N < fit ? N : fit);
    return p;
}
// Rows of the backward in flight: fewer than fit when that keeps the partial sums small
// beside the rows themselves.
NormPlan plan_bwd(long long N, int D, int num_sms)
{
    NormPlan p = plan_norm(N, D, num_sms, 512);
    const long long few = (N + 3) / 4;
    if (few < p.rows) p.rows = (int)few;
    return p;
}

template <typename Kernel>
cudaError_t launch(Kernel kern, const NormArgs &a, const NormPlan &p, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)p.rows * p.csize);
    cfg.blockDim = dim3(p.threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.csize;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.csize > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a, p.cols, p.csize);
}

template <typename E>
cudaError_t fwd_impl(const NormArgs &a, int num_sms, cudaStream_t stream)
{
    const NormPlan p = plan_norm(a.N, a.D, num_sms, 1024);
    if (a.D % 8 == 0)
        return p.csize > 1 ? launch(norm_fwd_kernel<E, true, true>, a, p, stream)
                           : launch(norm_fwd_kernel<E, true, false>, a, p, stream);
    return p.csize > 1 ? launch(norm_fwd_kernel<E, false, true>, a, p, stream)
                       : launch(norm_fwd_kernel<E, false, false>, a, p, stream);
}

template <typename E>
cudaError_t bwd_impl(const NormArgs &a, int num_sms, cudaStream_t stream)
{
    const NormPlan p = plan_bwd(a.N, a.D, num_sms);
    cudaError_t e;
    if (a.D % 8 == 0)
        e = p.csize > 1 ? launch(norm_bwd_kernel<E, true, true>, a, p, stream)
                        : launch(norm_bwd_kernel<E, true, false>, a, p, stream);
    else
        e = p.csize > 1 ? launch(norm_bwd_kernel<E, false, true>, a, p, stream)
                        : launch(norm_bwd_kernel<E, false, false>, a, p, stream);
    if (e != cudaSuccess) return e;
    norm_reduce_kernel<<<(a.D + 31) / 32, 256, 0, stream>>>(a, p.rows);
    return cudaGetLastError();
}

}  // namespace

size_t norm_bwd_partial_floats(long long N, int D, int num_sms) { return (size_t)plan_bwd(N, D, num_sms).rows * 2 * D; }

cudaError_t launch_norm_fwd(const NormArgs &a, bool bf16, int num_sms, cudaStream_t stream)
{
    return bf16 ? fwd_impl<__nv_bfloat16>(a, num_sms, stream) : fwd_impl<float>(a, num_sms, stream);
}

cudaError_t launch_norm_bwd(const NormArgs &a, bool bf16, int num_sms, cudaStream_t stream)
{
    return bf16 ? bwd_impl<__nv_bfloat16>(a, num_sms, stream) : bwd_impl<float>(a, num_sms, stream);
}

}  // namespace gdn2
