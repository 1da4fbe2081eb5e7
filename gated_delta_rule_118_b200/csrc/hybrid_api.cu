// hybrid_api.cu -- C ABI of the hybrid block's other operators: windowed
// attention with sinks, the gated linear recurrence and the block norm.  Checks
// of arguments, workspaces, and the launches on the caller's stream.
#include <cuda_runtime.h>

#include <math.h>
#include <stdint.h>

#include "gdn2.h"
#include "common.cuh"
#include "hybrid.h"
#include "launch.h"

using namespace gdn2;

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <int N>
gdn2_status check_required(const void *const (&ptrs)[N])
{
    for (const void *p : ptrs)
        if (!p) return GDN2_ERR_NULL;
    return GDN2_OK;
}

template <int N>
gdn2_status check_aligned(const void *const (&ptrs)[N])
{
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN2_ERR_ALIGN;
    return GDN2_OK;
}

bool dtype_ok(gdn2_dtype t) { return t == GDN2_F32 || t == GDN2_BF16; }
gdn2_status from_cuda(cudaError_t e) { return e == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA; }

// Element strides of one tensor whose axes have the given sizes (outermost
// first, rows of d elements), from the caller's (null: dense).
gdn2_status take_strides(const long long *given, const int *sizes, int n, int d, int esize, long long *out)
{
    long long dense = d;
    for (int i = n - 1; i >= 0; --i) {
        if (!given || sizes[i] <= 1) {
            out[i] = dense;
        } else {
            if (given[i] < d) return GDN2_ERR_SHAPE;
            if ((given[i] * esize) % 16 != 0) return GDN2_ERR_ALIGN;
            out[i] = given[i];
        }
        dense = out[i] * (sizes[i] > 1 ? sizes[i] : 1);
    }
    return GDN2_OK;
}

gdn2_status check_swa_sizes(int B, int Hq, int Hk, int d, int window, int sinks, float scale)
{
    if (B <= 0 || Hq <= 0 || Hk <= 0 || d <= 0 || window < 1 || sinks < 0) return GDN2_ERR_SHAPE;
    if (Hq % Hk != 0 || !(scale >= 1e-30f && scale <= 1e30f)) return GDN2_ERR_SHAPE;  // (lse / scale is formed)
    if (d != 64 && d != 128) return GDN2_ERR_UNSUPPORTED;
    if (B > 65535 || Hq > 65535) return GDN2_ERR_UNSUPPORTED;  // grid y/z limits
    return GDN2_OK;
}

gdn2_status swa_args(SwaArgs &a, const void *q, const void *k, const void *v, const int *lens, int B, int T, int Tk,
                     int Hq, int Hk, int d, int window, int sinks, float scale, const long long *strides,
                     gdn2_dtype dtype)
{
    if (!dtype_ok(dtype)) return GDN2_ERR_DTYPE;
    gdn2_status st = check_swa_sizes(B, Hq, Hk, d, window, sinks, scale);
    if (st != GDN2_OK) return st;
    if (T < 0 || Tk < T) return GDN2_ERR_SHAPE;
    if (Tk > GDN2_SWA_MAX_TOKENS) return GDN2_ERR_UNSUPPORTED;  // grid z limit
    const int esize = dtype == GDN2_BF16 ? 2 : 4;
    const int nq[3] = {B, T, Hq}, nk[3] = {B, Tk, Hk};
    if ((st = take_strides(strides, nq, 3, d, esize, a.qs)) != GDN2_OK) return st;
    if ((st = take_strides(strides ? strides + 3 : nullptr, nk, 3, d, esize, a.ks)) != GDN2_OK) return st;
    if ((st = take_strides(strides ? strides + 6 : nullptr, nk, 3, d, esize, a.vs)) != GDN2_OK) return st;
    a.q = q; a.k = k; a.v = v; a.lens = lens;
    a.B = B; a.T = T; a.Tk = Tk; a.Hq = Hq; a.Hk = Hk; a.d = d;
    a.window = window < Tk ? window : (Tk > 0 ? Tk : 1);
    a.sinks = sinks < Tk ? sinks : Tk;
    a.scale = scale;
    return GDN2_OK;
}

}  // namespace

extern "C" gdn2_status gdn2_swa_fwd(const void *q, const void *k, const void *v, const int *lens, void *o, float *lse,
                                    int B, int T, int Tk, int Hq, int Hk, int d, int window, int sinks, float scale,
                                    const long long *strides, gdn2_dtype dtype, gdn2_stream_t stream)
{
    SwaArgs a{};
    gdn2_status st = swa_args(a, q, k, v, lens, B, T, Tk, Hq, Hk, d, window, sinks, scale, strides, dtype);
    if (st != GDN2_OK) return st;
    if (T == 0) return GDN2_OK;
    if ((st = check_required({q, k, v, o})) != GDN2_OK) return st;
    if ((st = check_aligned({q, k, v, lens, o, lse})) != GDN2_OK) return st;
    a.out = o;
    a.lse = lse;
    int sms = 0;
    if (!device_info(&a.err, &sms)) return GDN2_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return from_cuda(dtype == GDN2_BF16 ? launch_swa_fwd_tc(a, s) : launch_swa_fwd_simt(a, s));
}

extern "C" gdn2_status gdn2_swa_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse,
                                    const void *dO, const int *lens, void *dq, void *dk, void *dv, int B, int T,
                                    int Tk, int Hq, int Hk, int d, int window, int sinks, float scale,
                                    const long long *strides, gdn2_dtype dtype, gdn2_stream_t stream)
{
    SwaArgs a{};
    gdn2_status st = swa_args(a, q, k, v, lens, B, T, Tk, Hq, Hk, d, window, sinks, scale, strides, dtype);
    if (st != GDN2_OK) return st;
    if (Tk == 0) return GDN2_OK;
    if ((st = check_required({dk, dv})) != GDN2_OK) return st;
    if ((st = check_aligned({q, k, v, o, lse, dO, lens, dq, dk, dv})) != GDN2_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int esize = dtype == GDN2_BF16 ? 2 : 4;
    if (T == 0) {  // no queries: dk = dv = 0
        const size_t bytes = (size_t)B * Tk * Hk * d * esize;
        cudaError_t e = cudaMemsetAsync(dk, 0, bytes, s);
        if (e == cudaSuccess) e = cudaMemsetAsync(dv, 0, bytes, s);
        return from_cuda(e);
    }
    if ((st = check_required({q, k, v, o, lse, dO, dq})) != GDN2_OK) return st;
    a.o = o; a.dO = dO; a.lse = const_cast<float *>(lse);
    a.dq = dq; a.dk = dk; a.dv = dv;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || !device_info(&a.err, &sms)) return GDN2_ERR_CUDA;
    cudaMemPool_t pool = workspace_pool(dev);
    if (!pool) return GDN2_ERR_CUDA;
    void *ws = nullptr;
    const bool tc = dtype == GDN2_BF16;
    const size_t rows = ((size_t)B * Hq * T + 3) / 4 * 4;  // (the partial sums behind delta stay 16-byte aligned)
    const size_t part = tc ? swa_bwd_tc_partial_floats(a, sms) : swa_bwd_simt_partial_floats(a, sms);
    if (cudaMallocFromPoolAsync(&ws, sizeof(float) * (rows + part), pool, s) != cudaSuccess) return GDN2_ERR_CUDA;
    a.delta = static_cast<float *>(ws);
    cudaError_t e = launch_swa_delta(a, tc, s);
    if (e == cudaSuccess)
        e = tc ? launch_swa_bwd_tc(a, a.delta + rows, sms, s) : launch_swa_bwd_simt(a, a.delta + rows, sms, s);
    const cudaError_t fe = cudaFreeAsync(ws, s);
    return from_cuda(e == cudaSuccess ? fe : e);
}

extern "C" gdn2_status gdn2_swa_decode(const void *q, const void *k, const void *v, void *k_cache, void *v_cache,
                                       const int *pos, void *o, int B, int slots, int Hq, int Hk, int d, int window,
                                       int sinks, float scale, const long long *strides, gdn2_dtype dtype,
                                       gdn2_stream_t stream)
{
    if (!dtype_ok(dtype)) return GDN2_ERR_DTYPE;
    gdn2_status st = check_swa_sizes(B, Hq, Hk, d, window, sinks, scale);
    if (st != GDN2_OK) return st;
    if ((long long)slots < (long long)sinks + window) return GDN2_ERR_SHAPE;
    if ((st = check_required({q, k, v, k_cache, v_cache, pos, o})) != GDN2_OK) return st;
    if ((st = check_aligned({q, k, v, k_cache, v_cache, pos, o})) != GDN2_OK) return st;
    SwaDecodeArgs a{};
    const int esize = dtype == GDN2_BF16 ? 2 : 4;
    const int nq[2] = {B, Hq}, nk[2] = {B, Hk};
    if ((st = take_strides(strides, nq, 2, d, esize, a.qs)) != GDN2_OK) return st;
    if ((st = take_strides(strides ? strides + 2 : nullptr, nk, 2, d, esize, a.ks)) != GDN2_OK) return st;
    if ((st = take_strides(strides ? strides + 4 : nullptr, nk, 2, d, esize, a.vs)) != GDN2_OK) return st;
    a.q = q; a.k = k; a.v = v; a.kc = k_cache; a.vc = v_cache; a.pos = pos; a.o = o;
    a.B = B; a.slots = slots; a.Hq = Hq; a.Hk = Hk; a.d = d; a.window = window; a.sinks = sinks; a.scale = scale;
    unsigned int *err = nullptr;
    int sms = 0;
    if (!device_info(&err, &sms)) return GDN2_ERR_CUDA;
    return from_cuda(launch_swa_decode(a, dtype == GDN2_BF16, sms, reinterpret_cast<cudaStream_t>(stream)));
}

namespace {

gdn2_status check_scan(int B, int T, int C, gdn2_dtype dtype)
{
    if (!dtype_ok(dtype)) return GDN2_ERR_DTYPE;
    if (B <= 0 || C <= 0 || T < 0) return GDN2_ERR_SHAPE;
    if (B > 65535) return GDN2_ERR_UNSUPPORTED;  // grid y limit
    return GDN2_OK;
}

}  // namespace

extern "C" gdn2_status gdn2_scan_fwd(const void *x, const void *w, const float *log_alpha, const float *h0, void *y,
                                     float *h_T, float *ckpt, int B, int T, int C, gdn2_dtype dtype,
                                     gdn2_stream_t stream)
{
    gdn2_status st = check_scan(B, T, C, dtype);
    if (st != GDN2_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if ((st = check_aligned({x, w, log_alpha, h0, y, h_T, ckpt})) != GDN2_OK) return st;
    if (T == 0) {  // nothing to run: h_T = h0 (or zeros)
        if (!h_T || h_T == h0) return GDN2_OK;
        const size_t bytes = sizeof(float) * (size_t)B * C;
        return from_cuda(h0 ? cudaMemcpyAsync(h_T, h0, bytes, cudaMemcpyDeviceToDevice, s)
                            : cudaMemsetAsync(h_T, 0, bytes, s));
    }
    if ((st = check_required({x, w, log_alpha, y})) != GDN2_OK) return st;
    ScanArgs a{};
    a.x = x; a.w = w; a.la = log_alpha; a.h0 = h0; a.y = y; a.h_T = h_T; a.ckpt = ckpt;
    a.B = B; a.T = T; a.C = C;
    unsigned int *err = nullptr;
    int sms = 0;
    if (!device_info(&err, &sms)) return GDN2_ERR_CUDA;
    a.err = err;
    return from_cuda(launch_scan_fwd(a, dtype == GDN2_BF16, sms, s));
}

extern "C" gdn2_status gdn2_scan_bwd(const void *x, const void *w, const float *log_alpha, const float *ckpt,
                                     const void *dy, const float *dh_T, void *dx, void *dw, float *dlog_alpha,
                                     float *dh0, int B, int T, int C, gdn2_dtype dtype, gdn2_stream_t stream)
{
    gdn2_status st = check_scan(B, T, C, dtype);
    if (st != GDN2_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if ((st = check_aligned({x, w, log_alpha, ckpt, dy, dh_T, dx, dw, dlog_alpha, dh0})) != GDN2_OK) return st;
    if (T == 0) {  // h_T = h0: dh0 = dh_T
        if (!dh0 || dh0 == dh_T) return GDN2_OK;
        const size_t bytes = sizeof(float) * (size_t)B * C;
        return from_cuda(dh_T ? cudaMemcpyAsync(dh0, dh_T, bytes, cudaMemcpyDeviceToDevice, s)
                              : cudaMemsetAsync(dh0, 0, bytes, s));
    }
    if ((st = check_required({x, w, log_alpha, ckpt, dy, dx, dw, dlog_alpha})) != GDN2_OK) return st;
    ScanArgs a{};
    a.x = x; a.w = w; a.la = log_alpha; a.ckpt = const_cast<float *>(ckpt); a.dy = dy; a.dh_T = dh_T;
    a.dx = dx; a.dw = dw; a.dla = dlog_alpha; a.dh0 = dh0;
    a.B = B; a.T = T; a.C = C;
    unsigned int *err = nullptr;
    int sms = 0;
    if (!device_info(&err, &sms)) return GDN2_ERR_CUDA;
    a.err = err;
    return from_cuda(launch_scan_bwd(a, dtype == GDN2_BF16, sms, s));
}

extern "C" gdn2_status gdn2_scan_step(const void *x, const void *w, const float *log_alpha, float *h, void *y, int B,
                                      int C, gdn2_dtype dtype, gdn2_stream_t stream)
{
    gdn2_status st = check_scan(B, 1, C, dtype);
    if (st != GDN2_OK) return st;
    if ((st = check_required({x, w, log_alpha, h, y})) != GDN2_OK) return st;
    if ((st = check_aligned({x, w, log_alpha, h, y})) != GDN2_OK) return st;
    ScanArgs a{};
    a.x = x; a.w = w; a.la = log_alpha; a.y = y;
    a.B = B; a.T = 1; a.C = C;
    return from_cuda(launch_scan_step(a, h, dtype == GDN2_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

namespace {

gdn2_status check_norm(long long N, int D, float eps, gdn2_dtype dtype)
{
    if (!dtype_ok(dtype)) return GDN2_ERR_DTYPE;
    if (N < 0 || D <= 0 || !(eps >= 0.f) || !isfinite(eps)) return GDN2_ERR_SHAPE;
    if (D > 16384) return GDN2_ERR_UNSUPPORTED;
    return GDN2_OK;
}

}  // namespace

extern "C" gdn2_status gdn2_block_norm_fwd(const void *r, const void *y, const void *g_logit, const float *w_post,
                                           const float *res_scale, const float *w_pre, float eps, void *r_out,
                                           void *x_out, long long N, int D, gdn2_dtype dtype, gdn2_stream_t stream)
{
    gdn2_status st = check_norm(N, D, eps, dtype);
    if (st != GDN2_OK) return st;
    if (N == 0) return GDN2_OK;
    if ((st = check_required({r, y, w_post, res_scale, w_pre, r_out, x_out})) != GDN2_OK) return st;
    if ((st = check_aligned({r, y, g_logit, w_post, res_scale, w_pre, r_out, x_out})) != GDN2_OK) return st;
    NormArgs a{};
    a.r = r; a.y = y; a.g = g_logit; a.w_post = w_post; a.res = res_scale; a.w_pre = w_pre; a.eps = eps;
    a.r_out = r_out; a.x_out = x_out; a.N = N; a.D = D;
    unsigned int *err = nullptr;
    int sms = 0;
    if (!device_info(&err, &sms)) return GDN2_ERR_CUDA;
    a.err = err;
    return from_cuda(launch_norm_fwd(a, dtype == GDN2_BF16, sms, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" gdn2_status gdn2_block_norm_bwd(const void *r, const void *y, const void *g_logit, const float *w_post,
                                           const float *res_scale, const float *w_pre, float eps,
                                           const void *dr_out, const void *dx_out, void *dr, void *dy, void *dg_logit,
                                           float *dw_post, float *dres_scale, float *dw_pre, long long N, int D,
                                           gdn2_dtype dtype, gdn2_stream_t stream)
{
    gdn2_status st = check_norm(N, D, eps, dtype);
    if (st != GDN2_OK) return st;
    if ((st = check_required({dw_post, dres_scale, dw_pre})) != GDN2_OK) return st;
    if ((st = check_aligned({r, y, g_logit, w_post, res_scale, w_pre, dr_out, dx_out, dr, dy, dg_logit, dw_post,
                             dres_scale, dw_pre})) != GDN2_OK)
        return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (N == 0) {
        const size_t bytes = sizeof(float) * (size_t)D;
        cudaError_t e = cudaMemsetAsync(dw_post, 0, bytes, s);
        if (e == cudaSuccess) e = cudaMemsetAsync(dres_scale, 0, bytes, s);
        if (e == cudaSuccess) e = cudaMemsetAsync(dw_pre, 0, bytes, s);
        return from_cuda(e);
    }
    if ((st = check_required({r, y, w_post, res_scale, w_pre, dr_out, dx_out, dr, dy})) != GDN2_OK) return st;
    if ((g_logit == nullptr) != (dg_logit == nullptr)) return GDN2_ERR_NULL;
    NormArgs a{};
    a.r = r; a.y = y; a.g = g_logit; a.w_post = w_post; a.res = res_scale; a.w_pre = w_pre; a.eps = eps;
    a.dr_out = dr_out; a.dx_out = dx_out; a.dr = dr; a.dy = dy; a.dg = dg_logit;
    a.dw_post = dw_post; a.dres = dres_scale; a.dw_pre = dw_pre; a.N = N; a.D = D;
    int dev = 0, sms = 0;
    unsigned int *err = nullptr;
    if (cudaGetDevice(&dev) != cudaSuccess || !device_info(&err, &sms)) return GDN2_ERR_CUDA;
    cudaMemPool_t pool = workspace_pool(dev);
    if (!pool) return GDN2_ERR_CUDA;
    void *ws = nullptr;
    if (cudaMallocFromPoolAsync(&ws, sizeof(float) * norm_bwd_partial_floats(N, D, dtype == GDN2_BF16, sms), pool, s) != cudaSuccess)
        return GDN2_ERR_CUDA;
    a.partial = static_cast<float *>(ws);
    a.err = err;
    const cudaError_t e = launch_norm_bwd(a, dtype == GDN2_BF16, sms, s);
    const cudaError_t fe = cudaFreeAsync(ws, s);
    return from_cuda(e == cudaSuccess ? fe : e);
}
