// block_norm.cu -- the norms around a block, fused with its gate and residual
// scale, forward and backward.  One CTA per row; every pass over the row reads
// it again (from cache).
#include "common.cuh"
#include "hybrid.h"

namespace gdn2 {
namespace {

constexpr int kThreads = 256;

template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N])
{
    __shared__ float red[N][kThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int o = 16; o; o >>= 1) v[n] += __shfl_xor_sync(~0u, v[n], o);
        if (lane == 0) red[n][warp] = v[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
        v[n] = 0.f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) v[n] += red[n][w];
    }
    __syncthreads();
}

__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

template <typename E>
struct Row {
    const E *r, *y, *g;
    __device__ __forceinline__ Row(const NormArgs &a, long long n)
        : r(static_cast<const E *>(a.r) + n * a.D), y(static_cast<const E *>(a.y) + n * a.D),
          g(a.g ? static_cast<const E *>(a.g) + n * a.D : nullptr) {}
    __device__ __forceinline__ float gate(int c) const { return g ? sigmoid(to_f32(g[c])) : 1.f; }
};

template <typename E>
__global__ void __launch_bounds__(kThreads) norm_fwd_kernel(const NormArgs a)
{
    const Row<E> in(a, blockIdx.x);
    E *ro = static_cast<E *>(a.r_out) + (long long)blockIdx.x * a.D, *xo = static_cast<E *>(a.x_out) + (long long)blockIdx.x * a.D;
    extern __shared__ float r1s[];
    float s[1] = {0.f};
    for (int c = threadIdx.x; c < a.D; c += kThreads) s[0] = fmaf(to_f32(in.y[c]), to_f32(in.y[c]), s[0]);
    block_sum(s);
    const float iy = rsqrtf(s[0] / a.D + a.eps);
    s[0] = 0.f;
    for (int c = threadIdx.x; c < a.D; c += kThreads) {
        const float r1 = fmaf(a.res[c] * a.w_post[c] * in.gate(c), to_f32(in.y[c]) * iy, to_f32(in.r[c]));
        r1s[c] = r1;
        s[0] = fmaf(r1, r1, s[0]);
        ro[c] = from_f32<E>(r1);
    }
    block_sum(s);
    const float ir = rsqrtf(s[0] / a.D + a.eps);
    for (int c = threadIdx.x; c < a.D; c += kThreads) xo[c] = from_f32<E>(r1s[c] * ir * a.w_pre[c]);
}

// Rows blockIdx.x, blockIdx.x + gridDim.x, ...; column sums in shared memory.
template <typename E>
__global__ void __launch_bounds__(kThreads) norm_bwd_kernel(const NormArgs a)
{
    extern __shared__ float acc[];  // [2][D]
    for (int c = threadIdx.x; c < 2 * a.D; c += kThreads) acc[c] = 0.f;
    for (long long n = blockIdx.x; n < a.N; n += gridDim.x) {
        const Row<E> in(a, n);
        const E *dro = static_cast<const E *>(a.dr_out) + n * a.D, *dxo = static_cast<const E *>(a.dx_out) + n * a.D;
        float s[1] = {0.f}, s2[2] = {0.f, 0.f};
        for (int c = threadIdx.x; c < a.D; c += kThreads) s[0] = fmaf(to_f32(in.y[c]), to_f32(in.y[c]), s[0]);
        block_sum(s);
        const float iy = rsqrtf(s[0] / a.D + a.eps);
        auto r1_of = [&](int c) {
            return fmaf(a.res[c] * a.w_post[c] * in.gate(c), to_f32(in.y[c]) * iy, to_f32(in.r[c]));
        };
        for (int c = threadIdx.x; c < a.D; c += kThreads) {
            const float r1 = r1_of(c);
            s2[0] = fmaf(r1, r1, s2[0]);
            s2[1] = fmaf(to_f32(dxo[c]) * a.w_pre[c], r1, s2[1]);
        }
        block_sum(s2);
        const float ir = rsqrtf(s2[0] / a.D + a.eps), mx = s2[1] / a.D * ir * ir;
        s[0] = 0.f;
        auto dr_of = [&](int c, float r1) {
            return fmaf(ir, fmaf(to_f32(dxo[c]), a.w_pre[c], -r1 * mx), to_f32(dro[c]));
        };
        for (int c = threadIdx.x; c < a.D; c += kThreads) {
            const float yh = to_f32(in.y[c]) * iy;
            s[0] = fmaf(dr_of(c, r1_of(c)) * a.res[c] * a.w_post[c] * in.gate(c), yh, s[0]);
        }
        block_sum(s);
        const float my = s[0] / a.D;
        for (int c = threadIdx.x; c < a.D; c += kThreads) {
            const float yh = to_f32(in.y[c]) * iy, gt = in.gate(c), t = a.res[c] * a.w_post[c], r1 = r1_of(c);
            const float dr = dr_of(c, r1), bsum = dr * gt * yh;
            acc[c] += bsum;
            acc[a.D + c] = fmaf(to_f32(dxo[c]), r1 * ir, acc[a.D + c]);
            static_cast<E *>(a.dr)[n * a.D + c] = from_f32<E>(dr);
            static_cast<E *>(a.dy)[n * a.D + c] = from_f32<E>(iy * fmaf(-yh, my, dr * t * gt));
            if (a.dg) static_cast<E *>(a.dg)[n * a.D + c] = from_f32<E>(bsum * t * (1.f - gt));
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.D; c += kThreads) a.partial[(long long)blockIdx.x * 2 * a.D + c] = acc[c];
}

__global__ void __launch_bounds__(256) norm_reduce_kernel(const NormArgs a, int rows)
{
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.D) return;
    float b = 0.f, p = 0.f;
    for (int r = 0; r < rows; ++r) {
        b += a.partial[(long long)r * 2 * a.D + c];
        p += a.partial[(long long)r * 2 * a.D + a.D + c];
    }
    a.dw_post[c] = b * a.res[c];
    a.dres[c] = b * a.w_post[c];
    a.dw_pre[c] = p;
}

int bwd_grid(long long N, int num_sms) { return (int)(N < num_sms ? N : num_sms); }

template <typename E>
cudaError_t fwd_impl(const NormArgs &a, cudaStream_t stream)
{
    if (a.N > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(norm_fwd_kernel<E>, cudaFuncAttributeMaxDynamicSharedMemorySize, 16384 * 4);
    if (e != cudaSuccess) return e;
    norm_fwd_kernel<E><<<(unsigned)a.N, kThreads, sizeof(float) * a.D, stream>>>(a);
    return cudaGetLastError();
}

template <typename E>
cudaError_t bwd_impl(const NormArgs &a, int num_sms, cudaStream_t stream)
{
    cudaError_t e = cudaFuncSetAttribute(norm_bwd_kernel<E>, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * 16384 * 4);
    if (e != cudaSuccess) return e;
    const int grid = bwd_grid(a.N, num_sms);
    norm_bwd_kernel<E><<<grid, kThreads, 2 * sizeof(float) * a.D, stream>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    norm_reduce_kernel<<<(a.D + 255) / 256, 256, 0, stream>>>(a, grid);
    return cudaGetLastError();
}

}  // namespace

size_t norm_bwd_partial_floats(long long N, int D, int num_sms) { return (size_t)bwd_grid(N, num_sms) * 2 * D; }

cudaError_t launch_norm_fwd(const NormArgs &a, bool bf16, int num_sms, cudaStream_t stream)
{
    return bf16 ? fwd_impl<__nv_bfloat16>(a, stream) : fwd_impl<float>(a, stream);
}

cudaError_t launch_norm_bwd(const NormArgs &a, bool bf16, int num_sms, cudaStream_t stream)
{
    return bf16 ? bwd_impl<__nv_bfloat16>(a, num_sms, stream) : bwd_impl<float>(a, num_sms, stream);
}

}  // namespace gdn2
