// block_norm.cu -- the norms around a block, fused with its gate and residual
// scale, forward and backward.
//
// A row stays in registers: 8 columns a thread, up to 512 threads a CTA, and rows of
// more than 4096 columns across a cluster of up to four CTAs that exchange their sums
// through distributed shared memory.  So every tensor is read and written once.  CTAs
// walk over rows with the grid's stride: the vectors (weights, scales) and the backward's
// column sums stay in registers.  Rows are fetched ahead into a ring in shared memory by
// bulk copies (rows whose length is not a multiple of 8 by plain loads): the row sums of
// one row (two in the forward, three in the backward) would otherwise leave the memory
// idle.  Bound by HBM: 32768 x 2048 bf16 with a gate, forward 112 us (6.0 TB/s), backward
// 213 us (5.0; three CTAs an SM, with the column sums in shared memory to fit their
// registers, leave room for fewer rows fetched ahead: 226 us).  Long rows are bound by the
// exchange of their sums: 8192 x 8192 forward 151 us (4.4 TB/s), backward 361 (3.0).
//
// The backward's sums over rows (for the three vectors' gradients) are added in a fixed
// order: each CTA over its rows, then a small kernel over the CTAs.  dw_post and
// dres_scale are the same sum times the other vector, so two sums are kept, not three.
#include <cooperative_groups.h>

#include "common.cuh"
#include "hybrid.h"
#include "launch.h"
#include "packed.cuh"
#include "sm100.cuh"

namespace gdn2 {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxThreads = 512;
constexpr int kMaxCols = 8 * kMaxThreads;  // columns of one CTA

// Eight elements of a row: contiguous ones from the ring, or one every NT columns from
// memory for rows that are not a multiple of 8 long.
template <typename E, bool VEC>
struct Eight {
    alignas(16) E e[8];
    __device__ __forceinline__ void from_ring(const uint8_t *row, int tid, bool on)
    {
        constexpr int W = sizeof(E) / 2;  // 16-byte words
#pragma unroll
        for (int w = 0; w < W; ++w)
            reinterpret_cast<uint4 *>(e)[w] =
                on ? reinterpret_cast<const uint4 *>(row + tid * 8 * sizeof(E))[w] : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void from_memory(const E *row, int c0, int tid, int nt, int cols)
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = c0 + tid + i * nt;
            e[i] = c < cols ? row[c] : from_f32<E>(0.f);
        }
    }
    __device__ __forceinline__ f2 operator[](int i) const { return pair_of(e + 2 * i); }  // pair i of 4
};

constexpr int kMaxStages = 4;

// The rows of NT tensors, fetched ahead.
template <typename E, int NT>
struct Ring {
    uint8_t *data;
    uint64_t *full;           // [stages]
    const void *const *src;   // [NT], null: absent
    int stages, tensor_bytes; // bytes of one tensor's slot
    int s = 0;
    uint32_t ph = 0;
    // (one thread) the columns [c0, cols) of row n into the slot of stage st
    __device__ __forceinline__ void fetch(int st, long long n, int D, int c0, int cols)
    {
        const uint32_t bytes = (uint32_t)(cols - c0) * sizeof(E);
        uint32_t present = 0;
#pragma unroll
        for (int k = 0; k < NT; ++k) present += src[k] != nullptr;
        sm100::mbar_arrive_expect_tx(full + st, present * bytes);
#pragma unroll
        for (int k = 0; k < NT; ++k)
            if (src[k])
                sm100::bulk_load(data + (st * NT + k) * tensor_bytes, static_cast<const E *>(src[k]) + n * D + c0, bytes,
                                 full + st);
    }
    // this stage's row is here (false: the wait gave up)
    __device__ __forceinline__ bool wait(unsigned int *err) const { return sm100::mbar_wait(full + s, ph, err); }
    // (one thread) everything asked for has landed, or its wait given up
    __device__ __forceinline__ void drain(unsigned int *err)
    {
        for (int i = 0; i < stages; ++i, next()) (void)wait(err);
    }
    __device__ __forceinline__ const uint8_t *slot(int k) const { return data + (s * NT + k) * tensor_bytes; }
    __device__ __forceinline__ void next()
    {
        if (++s == stages) {
            s = 0;
            ph ^= 1;
        }
    }
};

template <typename E, bool VEC>
__device__ __forceinline__ void store_eight(E *row, const f2 (&f)[4], int c0, int tid, int nt, int cols)
{
    if constexpr (VEC) {
        if (c0 + tid * 8 < cols) {
            if constexpr (sizeof(E) == 2) {
                *reinterpret_cast<uint4 *>(row + c0 + tid * 8) =
                    make_uint4(bf16_pair(f[0]), bf16_pair(f[1]), bf16_pair(f[2]), bf16_pair(f[3]));
            } else {
                *reinterpret_cast<ulonglong2 *>(row + c0 + tid * 8) = make_ulonglong2(f[0], f[1]);
                *reinterpret_cast<ulonglong2 *>(row + c0 + tid * 8 + 4) = make_ulonglong2(f[2], f[3]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 u = unpack2(f[i / 2]);
            if (c0 + tid + i * nt < cols) row[c0 + tid + i * nt] = from_f32<E>(i & 1 ? u.y : u.x);
        }
    }
}
template <bool VEC>
__device__ __forceinline__ int column(int c0, int tid, int nt, int i)
{
    return VEC ? c0 + tid * 8 + i : c0 + tid + i * nt;
}

// 1 / (1 + e), e = 2^(-x log2 e): both steps are accurate to about 2^-22, which the sums over
// rows need (a half-precision hyperbolic tangent would show in their gradients).  Also gives e,
// and raises `far` to the largest exponent's magnitude.
__device__ __forceinline__ f2 sigmoid2(f2 x, f2 &e, float &far)
{
    float2 t = unpack2(mul2(x, both(-1.4426950408889634f)));
    far = fmaxf(far, fmaxf(fabsf(t.x), fabsf(t.y)));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(t.y));
    e = pack2(t.x, t.y);
    t = unpack2(add2(e, both(1.f)));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(t.x));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(t.y));
    return pack2(t.x, t.y);
}
__device__ __forceinline__ f2 sigmoid2(f2 x)
{
    f2 e;
    float far = 0.f;
    return sigmoid2(x, e, far);
}
// e as a factor of 1 - sigmoid = e * sigmoid, where an exponent beyond 54 occurs: 0 where the
// sigmoid is 1 in double precision too, and short of infinity, which the 0 of a closed gate
// must not meet.  (A NaN stays in the sigmoid.)
__device__ __forceinline__ f2 bounded(f2 e)
{
    const float2 t = unpack2(e);
    return pack2(t.x < 0x1p-54f ? 0.f : fminf(t.x, 0x1p125f), t.y < 0x1p-54f ? 0.f : fminf(t.y, 0x1p125f));
}

// Sums of N values over the CTA (NW warps at most; absent ones leave zeros), and over
// the cluster with CL, left in every thread.  Slots alternate, so the next sum may start
// while slower threads still read this one.  False in a thread whose wait gave up.
template <int NW>
struct SumSlots {
    alignas(16) float warp[2][2][NW];  // [slot][value][warp]
    ulonglong2 cta[2][4];              // [slot][CTA of the cluster]: its values
    uint64_t landed[2];                // [slot]: every CTA's values are here
};
template <int NW, bool CL>
struct RowSums {
    SumSlots<NW> &sl;
    unsigned int *err;
    int slot = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ RowSums(SumSlots<NW> &slots, unsigned int *err_) : sl(slots), err(err_)
    {
        for (int i = threadIdx.x; i < 4 * NW; i += blockDim.x) (&sl.warp[0][0][0])[i] = 0.f;
        if (CL && threadIdx.x < 2) {
            sm100::mbar_init(sl.landed + threadIdx.x, 1);
            sm100::fence_mbar_init();
        }
        __syncthreads();
        if constexpr (CL) cg::this_cluster().sync();  // every CTA has started, its barriers set up
    }
    template <int N>
    __device__ __forceinline__ bool operator()(float (&v)[N])
    {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
        for (int o = 16; o; o >>= 1)
#pragma unroll
            for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(~0u, v[n], o);
        if constexpr (NW > 1) {
            if (lane == 0)
#pragma unroll
                for (int n = 0; n < N; ++n) sl.warp[slot][n][warp] = v[n];
            __syncthreads();
#pragma unroll
            for (int n = 0; n < N; ++n) {
                float4 t = *reinterpret_cast<const float4 *>(sl.warp[slot][n]);
#pragma unroll
                for (int w = 4; w < NW; w += 4) {
                    const float4 u = *reinterpret_cast<const float4 *>(sl.warp[slot][n] + w);
                    t = make_float4(t.x + u.x, t.y + u.y, t.z + u.z, t.w + u.w);
                }
                v[n] = (t.x + t.y) + (t.z + t.w);
            }
        }
        if constexpr (CL) {
            // each CTA sends its values to all: 16 bytes that signal the receiver's barrier (8192
            // x 8192 bf16 forward: 150 us, and 229 with a barrier of the whole cluster).  A CTA
            // that sends for the sum after next has this CTA's values of the next, sent when all
            // of its threads had read these.
            cg::cluster_group cluster = cg::this_cluster();
            const int size = cluster.num_blocks(), rank = cluster.block_rank();
            if (threadIdx.x == 0) sm100::mbar_arrive_expect_tx(sl.landed + slot, size * 16);
            if (threadIdx.x < size) {
                const ulonglong2 mine = make_ulonglong2(pack2(v[0], N > 1 ? v[N - 1] : 0.f), 0);
                sm100::st_async_16(sm100::peer_smem(&sl.cta[slot][rank], threadIdx.x), mine,
                                   sm100::peer_smem(sl.landed + slot, threadIdx.x));
            }
            if (__builtin_expect(!sm100::mbar_wait(sl.landed + slot, ph, err), 0)) return false;
            f2 t = 0;
            for (int c = 0; c < size; ++c) t = add2(t, sl.cta[slot][c].x);
            const float2 u = unpack2(t);
            v[0] = u.x;
            if constexpr (N > 1) v[1] = u.y;
            if (slot) ph ^= 1;
        }
        slot ^= 1;
        return true;
    }
};

// A thread whose wait gave up leaves the kernel (barriers do not count threads that have left;
// what it no longer asks for, sends or signals lets the others' waits give up in turn), once
// the rows it asked for have landed and no sum is on its way to its CTA.
template <bool VEC, bool CL, typename R>
__device__ __forceinline__ void leave(R &ring, unsigned int *err)
{
    if (VEC && threadIdx.x == 0) ring.drain(err);
    if (CL) sm100::leave_cluster();
}

// CTAs of an SM that the register budget is set for: short rows have many small CTAs.
constexpr int fwd_ctas(int nw) { return nw == 1 ? 24 : nw == 4 ? 8 : nw == 8 ? 4 : 2; }
constexpr int bwd_ctas(int nw) { return nw == 1 ? 16 : nw == 4 ? 4 : nw == 8 ? 2 : 1; }

// The two vectors a row is multiplied with, in shared memory: res_scale * w_post, and w_pre.
template <bool VEC>
__device__ __forceinline__ void stage_vectors(float *vec, const NormArgs &a, int c0, int cols)
{
    const int n = cols - c0;
    for (int c = threadIdx.x; c < n; c += blockDim.x) {
        vec[c] = a.res[c0 + c] * a.w_post[c0 + c];
        vec[n + c] = a.w_pre[c0 + c];
    }
    __syncthreads();
}
template <bool VEC>
__device__ __forceinline__ void take_eight(f2 (&f)[4], const float *vec, int tid, int nt, int n)
{
    if constexpr (VEC) {
        const bool on = tid * 8 < n;
        const ulonglong2 z = make_ulonglong2(0, 0);
        const ulonglong2 u = on ? *reinterpret_cast<const ulonglong2 *>(vec + tid * 8) : z;
        const ulonglong2 w = on ? *reinterpret_cast<const ulonglong2 *>(vec + tid * 8 + 4) : z;
        f[0] = u.x; f[1] = u.y; f[2] = w.x; f[3] = w.y;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = tid + 2 * i * nt;
            f[i] = pack2(c < n ? vec[c] : 0.f, c + nt < n ? vec[c + nt] : 0.f);
        }
    }
}

template <typename E, bool VEC, bool CL, int NW>
__global__ void __launch_bounds__(32 * NW, fwd_ctas(NW)) norm_fwd_kernel(const NormArgs a, int cols_per_cta, int csize, int stages)
{
    __shared__ SumSlots<NW> slots;
    RowSums<NW, CL> sums(slots, a.err);
    const int tid = threadIdx.x, nt = blockDim.x;
    const int c0 = CL ? (int)(blockIdx.x % csize) * cols_per_cta : 0, cols = min(a.D, c0 + cols_per_cta);
    const long long first = blockIdx.x / csize, step = gridDim.x / csize;
    const float rd = 1.f / a.D;
    extern __shared__ __align__(128) uint8_t dyn[];
    float *vec = reinterpret_cast<float *>(dyn);
    uint8_t *ring_data = dyn + 8 * cols_per_cta;
    __shared__ __align__(8) uint64_t full[kMaxStages];
    stage_vectors<VEC>(vec, a, c0, cols);
    const void *const src[3] = {a.y, a.r, a.g};
    Ring<E, 3> ring{ring_data, full, src, stages, cols_per_cta * (int)sizeof(E)};
    Eight<E, VEC> y, r, g;
    if constexpr (VEC) {
        if (tid == 0) {
            for (int s = 0; s < stages; ++s) sm100::mbar_init(full + s, 1);
            sm100::fence_mbar_init();
            for (int s = 0; s < stages; ++s)
                if (first + s * step < a.N) ring.fetch(s, first + s * step, a.D, c0, cols);
        }
        __syncthreads();
    }
    for (long long n = first; n < a.N; n += step) {
        if constexpr (VEC) {
            const bool on = c0 + tid * 8 < cols;
            if (__builtin_expect(!ring.wait(a.err), 0)) return leave<VEC, CL>(ring, a.err);
            y.from_ring(ring.slot(0), tid, on);
            r.from_ring(ring.slot(1), tid, on);
            g.from_ring(ring.slot(2), tid, on);
        } else {
            y.from_memory(static_cast<const E *>(a.y) + n * a.D, c0, tid, nt, cols);
            r.from_memory(static_cast<const E *>(a.r) + n * a.D, c0, tid, nt, cols);
            if (a.g) g.from_memory(static_cast<const E *>(a.g) + n * a.D, c0, tid, nt, cols);
        }
        f2 yv[4], r1[4], gt[4], sq = 0;
        take_eight<VEC>(gt, vec, tid, nt, cols - c0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            yv[i] = y[i];
            r1[i] = r[i];
            if (a.g) gt[i] = mul2(gt[i], sigmoid2(g[i]));
            sq = fma2(yv[i], yv[i], sq);
        }
        float s[1] = {sum2(sq)};
        if (__builtin_expect(!sums(s), 0)) return leave<VEC, CL>(ring, a.err);
        if constexpr (VEC) {  // every thread has its columns: the slot takes the row `stages` ahead
            if constexpr (NW == 1) __syncwarp();
            if (tid == 0 && n + stages * step < a.N) ring.fetch(ring.s, n + stages * step, a.D, c0, cols);
            ring.next();
        }
        const f2 iy = both(rsqrtf(fmaf(s[0], rd, a.eps)));
        sq = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r1[i] = fma2(gt[i], mul2(yv[i], iy), r1[i]);
            sq = fma2(r1[i], r1[i], sq);
        }
        store_eight<E, VEC>(static_cast<E *>(a.r_out) + n * a.D, r1, c0, tid, nt, cols);
        s[0] = sum2(sq);
        if (__builtin_expect(!sums(s), 0)) return leave<VEC, CL>(ring, a.err);
        const f2 ir = both(rsqrtf(fmaf(s[0], rd, a.eps)));
        f2 wq[4];
        take_eight<VEC>(wq, vec + cols - c0, tid, nt, cols - c0);
#pragma unroll
        for (int i = 0; i < 4; ++i) r1[i] = mul2(r1[i], mul2(ir, wq[i]));
        store_eight<E, VEC>(static_cast<E *>(a.x_out) + n * a.D, r1, c0, tid, nt, cols);
    }
    // (nothing is on its way to a CTA here: it has waited for each of its sums and rows)
}

template <typename E, bool VEC, bool CL, int NW>
__global__ void __launch_bounds__(32 * NW, bwd_ctas(NW)) norm_bwd_kernel(const NormArgs a, int cols_per_cta, int csize, int stages)
{
    __shared__ SumSlots<NW> slots;
    RowSums<NW, CL> sums(slots, a.err);
    const int tid = threadIdx.x, nt = blockDim.x;
    const int c0 = CL ? (int)(blockIdx.x % csize) * cols_per_cta : 0, cols = min(a.D, c0 + cols_per_cta);
    const long long first = blockIdx.x / csize, step = gridDim.x / csize;
    const float rd = 1.f / a.D;
    f2 bsum[4] = {}, psum[4] = {};
    extern __shared__ __align__(128) uint8_t dyn[];
    float *vec = reinterpret_cast<float *>(dyn);
    uint8_t *ring_data = dyn + 8 * cols_per_cta;
    __shared__ __align__(8) uint64_t full[kMaxStages];
    stage_vectors<VEC>(vec, a, c0, cols);
    const void *const src[5] = {a.y, a.r, a.g, a.dx_out, a.dr_out};
    Ring<E, 5> ring{ring_data, full, src, stages, cols_per_cta * (int)sizeof(E)};
    Eight<E, VEC> y, r, g, dx, dr;
    if constexpr (VEC) {
        if (tid == 0) {
            for (int s = 0; s < stages; ++s) sm100::mbar_init(full + s, 1);
            sm100::fence_mbar_init();
            for (int s = 0; s < stages; ++s)
                if (first + s * step < a.N) ring.fetch(s, first + s * step, a.D, c0, cols);
        }
        __syncthreads();
    }
    for (long long n = first; n < a.N; n += step) {
        if constexpr (VEC) {
            const bool on = c0 + tid * 8 < cols;
            if (__builtin_expect(!ring.wait(a.err), 0)) return leave<VEC, CL>(ring, a.err);
            y.from_ring(ring.slot(0), tid, on);
            r.from_ring(ring.slot(1), tid, on);
            g.from_ring(ring.slot(2), tid, on);
            dx.from_ring(ring.slot(3), tid, on);
            dr.from_ring(ring.slot(4), tid, on);
        } else {
            y.from_memory(static_cast<const E *>(a.y) + n * a.D, c0, tid, nt, cols);
            r.from_memory(static_cast<const E *>(a.r) + n * a.D, c0, tid, nt, cols);
            if (a.g) g.from_memory(static_cast<const E *>(a.g) + n * a.D, c0, tid, nt, cols);
            dx.from_memory(static_cast<const E *>(a.dx_out) + n * a.D, c0, tid, nt, cols);
            dr.from_memory(static_cast<const E *>(a.dr_out) + n * a.D, c0, tid, nt, cols);
        }
        f2 yv[4], r1[4], gt[4], ge[4], xv[4], dv[4], sq = 0, sx = 0;
        float far = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            yv[i] = y[i];
            r1[i] = r[i];
            gt[i] = a.g ? sigmoid2(g[i], ge[i], far) : both(1.f);
            xv[i] = dx[i];
            dv[i] = dr[i];
            sq = fma2(yv[i], yv[i], sq);
        }
        if (__builtin_expect(far > 54.f, 0)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) ge[i] = bounded(ge[i]);
        }
        // 1 - gate as e * gate: the difference has 3 % of itself left at a logit of 12, and nothing
        // above 17.  (Formed here, or at its use where registers are short: 30000 x 1001 bf16 231
        // us, and 249 formed here; 16384 x 4096 fp32 368 formed here, and 388 at its use.)
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < 4; ++i) ge[i] = mul2(ge[i], gt[i]);
        }
        float s[1] = {sum2(sq)};
        if (__builtin_expect(!sums(s), 0)) return leave<VEC, CL>(ring, a.err);
        if constexpr (VEC) {  // every thread has its columns: the slot takes the row `stages` ahead
            if constexpr (NW == 1) __syncwarp();
            if (tid == 0 && n + stages * step < a.N) ring.fetch(ring.s, n + stages * step, a.D, c0, cols);
            ring.next();
        }
        const f2 iy = both(rsqrtf(fmaf(s[0], rd, a.eps)));
        f2 t[4], wx[4];
        take_eight<VEC>(t, vec, tid, nt, cols - c0);
        take_eight<VEC>(wx, vec + cols - c0, tid, nt, cols - c0);
        sq = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            yv[i] = mul2(yv[i], iy);
            r1[i] = fma2(mul2(t[i], gt[i]), yv[i], r1[i]);
            wx[i] = mul2(wx[i], xv[i]);
            sq = fma2(r1[i], r1[i], sq);
            sx = fma2(wx[i], r1[i], sx);
        }
        float q[2] = {sum2(sq), sum2(sx)};
        if (__builtin_expect(!sums(q), 0)) return leave<VEC, CL>(ring, a.err);
        const float irs = rsqrtf(fmaf(q[0], rd, a.eps));
        const f2 ir = both(irs), mx = both(-q[1] * rd * irs * irs);
        sq = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            dv[i] = fma2(ir, fma2(mx, r1[i], wx[i]), dv[i]);
            psum[i] = fma2(xv[i], mul2(r1[i], ir), psum[i]);
            xv[i] = mul2(dv[i], gt[i]);       // gradient of the gated term, before its scale
            r1[i] = mul2(xv[i], t[i]);
            sq = fma2(r1[i], yv[i], sq);
        }
        store_eight<E, VEC>(static_cast<E *>(a.dr) + n * a.D, dv, c0, tid, nt, cols);
        s[0] = sum2(sq);
        if (__builtin_expect(!sums(s), 0)) return leave<VEC, CL>(ring, a.err);
        const f2 my = both(-s[0] * rd);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f2 b = mul2(xv[i], yv[i]), bt = mul2(b, t[i]);
            bsum[i] = add2(bsum[i], b);
            r1[i] = mul2(iy, fma2(my, yv[i], r1[i]));
            if (a.g) dv[i] = mul2(bt, VEC ? ge[i] : mul2(ge[i], gt[i]));
        }
        store_eight<E, VEC>(static_cast<E *>(a.dy) + n * a.D, r1, c0, tid, nt, cols);
        if (a.g) store_eight<E, VEC>(static_cast<E *>(a.dg) + n * a.D, dv, c0, tid, nt, cols);
    }
    float *part = a.partial + first * 2 * a.D;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = column<VEC>(c0, tid, nt, i);
        const float2 bs = unpack2(bsum[i / 2]), ps = unpack2(psum[i / 2]);
        if (c < cols) {
            part[c] = i & 1 ? bs.y : bs.x;
            part[a.D + c] = i & 1 ? ps.y : ps.x;
        }
    }
}

// 32 columns a CTA, its 32 warps over the partial rows: many loads in flight, since each
// row is one 128-byte line.
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const NormArgs a, int rows)
{
    __shared__ float red[2][32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float b = 0.f, p = 0.f;
    if (c < a.D) {
#pragma unroll 8
        for (int r = warp; r < rows; r += 32) {
            b += a.partial[(long long)r * 2 * a.D + c];
            p += a.partial[(long long)r * 2 * a.D + a.D + c];
        }
    }
    red[0][warp][lane] = b;
    red[1][warp][lane] = p;
    __syncthreads();
    if (warp == 0 && c < a.D) {
        b = p = 0.f;
#pragma unroll
        for (int w = 0; w < 32; ++w) {
            b += red[0][w][lane];
            p += red[1][w][lane];
        }
        a.dw_post[c] = b * a.res[c];
        a.dres[c] = b * a.w_post[c];
        a.dw_pre[c] = p;
    }
}

// CTAs of the cluster, columns and threads of each, rows in flight, and the ring.
struct NormPlan {
    int csize, cols, threads, nw, rows, stages, smem;
};
NormPlan plan_norm(long long N, int D, int num_sms, int (*ctas)(int), int row_bytes_per_col)
{
    NormPlan p;
    p.csize = D <= kMaxCols ? 1 : D <= 2 * kMaxCols ? 2 : 4;
    p.cols = (D + p.csize - 1) / p.csize;
    p.cols = (p.cols + 7) / 8 * 8;
    p.threads = (p.cols + 255) / 256 * 32;
    p.nw = p.threads <= 32 ? 1 : p.threads <= 128 ? 4 : p.threads <= 256 ? 8 : 16;
    const int per_sm = ctas(p.nw);
    const long long fit = (long long)num_sms * per_sm / p.csize;
    p.rows = (int)(N < fit ? N : fit);
    const int vec = 8 * p.cols, slot = p.cols * row_bytes_per_col, room = 208 * 1024 / per_sm - 1024 - vec;
    p.stages = room / slot > kMaxStages ? kMaxStages : room / slot < 1 ? 1 : room / slot;
    p.smem = vec + (D % 8 == 0 ? p.stages * slot : 0);
    return p;
}
NormPlan plan_fwd(long long N, int D, int num_sms, int esize) { return plan_norm(N, D, num_sms, fwd_ctas, 3 * esize); }
// Rows of the backward in flight: fewer than fit when that keeps the partial sums small
// beside the rows themselves.
NormPlan plan_bwd(long long N, int D, int num_sms, int esize)
{
    NormPlan p = plan_norm(N, D, num_sms, bwd_ctas, 5 * esize);
    const long long few = (N + 3) / 4;
    if (few < p.rows) p.rows = (int)few;
    return p;
}

template <auto kern>
cudaError_t launch(const NormArgs &a, const NormPlan &p, cudaStream_t stream)
{
    static std::atomic<unsigned long long> set{0};
    cudaError_t e = ensure_smem_limit(kern, 208 * 1024, set);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)p.rows * p.csize);
    cfg.blockDim = dim3(p.threads);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.csize;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.csize > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a, p.cols, p.csize, p.stages);
}

template <typename E, bool VEC>
cudaError_t fwd_rows(const NormArgs &a, const NormPlan &p, cudaStream_t stream)
{
    if (p.csize > 1) return launch<norm_fwd_kernel<E, VEC, true, 16>>(a, p, stream);
    switch (p.nw) {
    case 1: return launch<norm_fwd_kernel<E, VEC, false, 1>>(a, p, stream);
    case 4: return launch<norm_fwd_kernel<E, VEC, false, 4>>(a, p, stream);
    case 8: return launch<norm_fwd_kernel<E, VEC, false, 8>>(a, p, stream);
    default: return launch<norm_fwd_kernel<E, VEC, false, 16>>(a, p, stream);
    }
}
template <typename E, bool VEC>
cudaError_t bwd_rows(const NormArgs &a, const NormPlan &p, cudaStream_t stream)
{
    if (p.csize > 1) return launch<norm_bwd_kernel<E, VEC, true, 16>>(a, p, stream);
    switch (p.nw) {
    case 1: return launch<norm_bwd_kernel<E, VEC, false, 1>>(a, p, stream);
    case 4: return launch<norm_bwd_kernel<E, VEC, false, 4>>(a, p, stream);
    case 8: return launch<norm_bwd_kernel<E, VEC, false, 8>>(a, p, stream);
    default: return launch<norm_bwd_kernel<E, VEC, false, 16>>(a, p, stream);
    }
}

template <typename E>
cudaError_t fwd_impl(const NormArgs &a, int num_sms, cudaStream_t stream)
{
    const NormPlan p = plan_fwd(a.N, a.D, num_sms, sizeof(E));
    return a.D % 8 == 0 ? fwd_rows<E, true>(a, p, stream) : fwd_rows<E, false>(a, p, stream);
}

template <typename E>
cudaError_t bwd_impl(const NormArgs &a, int num_sms, cudaStream_t stream)
{
    const NormPlan p = plan_bwd(a.N, a.D, num_sms, sizeof(E));
    const cudaError_t e = a.D % 8 == 0 ? bwd_rows<E, true>(a, p, stream) : bwd_rows<E, false>(a, p, stream);
    if (e != cudaSuccess) return e;
    return launch_plain(norm_reduce_kernel, dim3((a.D + 31) / 32), dim3(1024), 0, stream, a, p.rows);
}

}  // namespace

size_t norm_bwd_partial_floats(long long N, int D, bool bf16, int num_sms)
{
    return (size_t)plan_bwd(N, D, num_sms, bf16 ? 2 : 4).rows * 2 * D;
}

cudaError_t launch_norm_fwd(const NormArgs &a, bool bf16, int num_sms, cudaStream_t stream)
{
    return bf16 ? fwd_impl<__nv_bfloat16>(a, num_sms, stream) : fwd_impl<float>(a, num_sms, stream);
}

cudaError_t launch_norm_bwd(const NormArgs &a, bool bf16, int num_sms, cudaStream_t stream)
{
    return bf16 ? bwd_impl<__nv_bfloat16>(a, num_sms, stream) : bwd_impl<float>(a, num_sms, stream);
}

}  // namespace gdn2
