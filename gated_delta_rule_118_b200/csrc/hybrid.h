// hybrid.h -- internal (C++) interface between the C ABI layer and the kernels of
// the hybrid block's other operators (windowed attention, gated linear
// recurrence, block norm).  Arguments arrive here already validated by
// hybrid_api.cu.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn2 {

// Windowed attention.  window and sinks are cut to Tk; strides are in elements.
struct SwaArgs {
    const void *q, *k, *v, *o, *dO;  // o: the forward's output (backward only)
    const int *lens;                 // may be null
    void *out;                       // forward output
    float *lse;                      // may be null in the forward
    void *dq, *dk, *dv;
    float *delta;                    // [B][Hq][T] workspace of the backward: dO . o
    long long qs[3], ks[3], vs[3];   // {batch, token, head}
    int B, T, Tk, Hq, Hk, d, window, sinks;
    float scale;
    unsigned int *err;               // device error word
};
cudaError_t launch_swa_fwd_simt(const SwaArgs &a, cudaStream_t stream);     // fp32
cudaError_t launch_swa_fwd_tc(const SwaArgs &a, cudaStream_t stream);  // bf16
// Backward; `part`: ..._partial_floats(...) of workspace for partial sums of dk and dv.
size_t swa_bwd_simt_partial_floats(const SwaArgs &a, int num_sms);
cudaError_t launch_swa_bwd_simt(const SwaArgs &a, float *part, int num_sms, cudaStream_t stream);  // fp32
size_t swa_bwd_tc_partial_floats(const SwaArgs &a, int num_sms);
cudaError_t launch_swa_bwd_tc(const SwaArgs &a, float *part, int num_sms, cudaStream_t stream);    // bf16
cudaError_t launch_swa_delta(const SwaArgs &a, bool bf16, cudaStream_t stream);

struct SwaDecodeArgs {
    const void *q, *k, *v;
    void *kc, *vc;
    const int *pos;
    void *o;
    long long qs[2], ks[2], vs[2];   // {batch, head}
    int B, slots, Hq, Hk, d, window, sinks;
    float scale;
};
cudaError_t launch_swa_decode(const SwaDecodeArgs &a, bool bf16, int num_sms, cudaStream_t stream);

// Gated linear recurrence over [B][T][C].
constexpr int kScanBlock = 16;       // tokens between checkpoints (GDN2_SCAN_BLOCK)
struct ScanArgs {
    const void *x, *w;
    const float *la;
    const float *h0;                 // may be null
    void *y;
    float *h_T;                      // may be null
    float *ckpt;                     // may be null (forward)
    const void *dy;
    const float *dh_T;               // may be null
    void *dx, *dw;
    float *dla;
    float *dh0;                      // may be null
    int B, T, C;
    unsigned int *err;               // device error word
};
cudaError_t launch_scan_fwd(const ScanArgs &a, bool bf16, int num_sms, cudaStream_t stream);
cudaError_t launch_scan_bwd(const ScanArgs &a, bool bf16, int num_sms, cudaStream_t stream);
cudaError_t launch_scan_step(const ScanArgs &a, float *h, bool bf16, cudaStream_t stream);

// Block norm over N rows of D channels.
struct NormArgs {
    const void *r, *y, *g;           // g may be null
    const float *w_post, *res, *w_pre;
    float eps;
    void *r_out, *x_out;
    const void *dr_out, *dx_out;
    void *dr, *dy, *dg;
    float *dw_post, *dres, *dw_pre;
    float *partial;                  // norm_bwd_partial_floats(...) of workspace
    long long N;
    int D;
    unsigned int *err;               // device error word
};
cudaError_t launch_norm_fwd(const NormArgs &a, bool bf16, int num_sms, cudaStream_t stream);
size_t norm_bwd_partial_floats(long long N, int D, bool bf16, int num_sms);
cudaError_t launch_norm_bwd(const NormArgs &a, bool bf16, int num_sms, cudaStream_t stream);

}  // namespace gdn2
