// scan.cu -- the gated linear recurrence h_t = alpha_t h_{t-1} + w_t x_t per
// channel: forward, backward and single step.  One thread per (batch, channel)
// walks the tokens; bound by the latency of its loads when there are few channels.
#include "common.cuh"
#include "hybrid.h"

namespace gdn2 {
namespace {

constexpr int kThreads = 64;

template <typename E>
__global__ void __launch_bounds__(kThreads) scan_fwd_kernel(const ScanArgs a)
{
    const int c = blockIdx.x * kThreads + threadIdx.x, b = blockIdx.y;
    if (c >= a.C) return;
    const long long row0 = (long long)b * a.T * a.C + c;
    const int nblk = (a.T + kScanBlock - 1) / kScanBlock;
    float h = a.h0 ? a.h0[(long long)b * a.C + c] : 0.f;
    for (int blk = 0; blk < nblk; ++blk) {
        if (a.ckpt) a.ckpt[((long long)b * nblk + blk) * a.C + c] = h;
        float la[kScanBlock], u[kScanBlock];
#pragma unroll
        for (int t = 0; t < kScanBlock; ++t) {
            const bool on = blk * kScanBlock + t < a.T;
            const long long i = row0 + (long long)(blk * kScanBlock + t) * a.C;
            la[t] = on ? a.la[i] : 0.f;
            u[t] = on ? to_f32(static_cast<const E *>(a.x)[i]) * to_f32(static_cast<const E *>(a.w)[i]) : 0.f;
        }
#pragma unroll
        for (int t = 0; t < kScanBlock; ++t) {
            if (blk * kScanBlock + t >= a.T) break;
            h = fmaf(expf(la[t]), h, u[t]);
            static_cast<E *>(a.y)[row0 + (long long)(blk * kScanBlock + t) * a.C] = from_f32<E>(h);
        }
    }
    if (a.h_T) a.h_T[(long long)b * a.C + c] = h;
}

template <typename E>
__global__ void __launch_bounds__(kThreads) scan_bwd_kernel(const ScanArgs a)
{
    const int c = blockIdx.x * kThreads + threadIdx.x, b = blockIdx.y;
    if (c >= a.C) return;
    const long long row0 = (long long)b * a.T * a.C + c;
    const int nblk = (a.T + kScanBlock - 1) / kScanBlock;
    float g = a.dh_T ? a.dh_T[(long long)b * a.C + c] : 0.f;  // gradient of h_t from later tokens
    for (int blk = nblk - 1; blk >= 0; --blk) {
        float al[kScanBlock], x[kScanBlock], w[kScanBlock], hp[kScanBlock];
        float h = a.ckpt[((long long)b * nblk + blk) * a.C + c];
#pragma unroll
        for (int t = 0; t < kScanBlock; ++t) {
            const bool on = blk * kScanBlock + t < a.T;
            const long long i = row0 + (long long)(blk * kScanBlock + t) * a.C;
            al[t] = on ? expf(a.la[i]) : 1.f;
            x[t] = on ? to_f32(static_cast<const E *>(a.x)[i]) : 0.f;
            w[t] = on ? to_f32(static_cast<const E *>(a.w)[i]) : 0.f;
        }
#pragma unroll
        for (int t = 0; t < kScanBlock; ++t) {
            hp[t] = h;
            h = fmaf(al[t], h, w[t] * x[t]);
        }
#pragma unroll
        for (int t = kScanBlock - 1; t >= 0; --t) {
            if (blk * kScanBlock + t >= a.T) continue;
            const long long i = row0 + (long long)(blk * kScanBlock + t) * a.C;
            g += to_f32(static_cast<const E *>(a.dy)[i]);
            static_cast<E *>(a.dx)[i] = from_f32<E>(g * w[t]);
            static_cast<E *>(a.dw)[i] = from_f32<E>(g * x[t]);
            g *= al[t];
            a.dla[i] = g * hp[t];
        }
    }
    if (a.dh0) a.dh0[(long long)b * a.C + c] = g;
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

}  // namespace

cudaError_t launch_scan_fwd(const ScanArgs &a, bool bf16, int num_sms, cudaStream_t stream)
{
    const dim3 grid((a.C + kThreads - 1) / kThreads, a.B);
    if (bf16) scan_fwd_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(a);
    else scan_fwd_kernel<float><<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_scan_bwd(const ScanArgs &a, bool bf16, int num_sms, cudaStream_t stream)
{
    const dim3 grid((a.C + kThreads - 1) / kThreads, a.B);
    if (bf16) scan_bwd_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(a);
    else scan_bwd_kernel<float><<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_scan_step(const ScanArgs &a, float *h, bool bf16, cudaStream_t stream)
{
    const long long blocks = ((long long)a.B * a.C + 255) / 256;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (bf16) scan_step_kernel<__nv_bfloat16><<<(unsigned)blocks, 256, 0, stream>>>(a, h);
    else scan_step_kernel<float><<<(unsigned)blocks, 256, 0, stream>>>(a, h);
    return cudaGetLastError();
}

}  // namespace gdn2
