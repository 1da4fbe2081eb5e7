// swa_simt.cu -- windowed attention in fp32 on the CUDA cores: forward, and the
// backward as two kernels without atomics (dq by query tiles; dk and dv by key
// tiles).  The products are 64-wide register tiles over shared memory; bound by
// the FFMA rate (every score costs 2 d FMAs, and the two-kernel backward forms
// q k^T and dO v^T twice in exchange for a fixed order of every sum).  3 x 333 x 6 heads
// of 64 over 2, window 100, forward and backward: 121 us in five launches, each a fraction
// of a wave, so bound by the walk of one CTA; 2 x 4096 x 8 heads of 64, window 512: forward
// 342 us, backward 2010, a third and a fifth of the FFMA rate: a dot product's register tile
// of 4 x 4 reads shared memory for three quarters of its FMAs' cycles, the backward's of 4 x 2
// and 2 x 4 for as many cycles as its FMAs, and three to five barriers a tile stand between.
#include "launch.h"
#include "swa_common.cuh"

namespace gdn2 {
namespace {

using namespace swa;

constexpr int kThreads = 256;  // 16 x 16: ty = query (or key) rows, tx = columns

// Rows [r0, r0 + N) of `src` into shared memory (row stride D + 4), zeros from row `end` on.
template <typename E, int D, int N>
__device__ __forceinline__ void load_rows(float *dst, const Rows<E> &src, int r0, int end)
{
    for (int c = threadIdx.x; c < N * D / 4; c += kThreads) {
        const int r = c / (D / 4), x = c % (D / 4) * 4;
        const float4 f = r0 + r < end ? load4(src[r0 + r] + x) : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4 *>(dst + r * (D + 4) + x) = f;
    }
}

// The same without waiting: copies of one group, ended by rows_asked.
template <typename E, int D, int N>
__device__ __forceinline__ void ask_rows(float *dst, const Rows<E> &src, int r0, int end)
{
    static_assert(sizeof(E) == 4, "rows are copied as they are");
#pragma unroll
    for (int c = threadIdx.x; c < N * D / 4; c += kThreads) {
        const int r = c / (D / 4), x = c % (D / 4) * 4;
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst + r * (D + 4) + x);
        const int bytes = r0 + r < end ? 16 : 0;  // (the rest of the 16 is filled with zeros)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src[min(r0 + r, end - 1)] + x), "r"(bytes) : "memory");
    }
}
__device__ __forceinline__ void rows_asked() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LATER>
__device__ __forceinline__ void rows_landed()  // all groups but the last LATER
{
    asm volatile("cp.async.wait_group %0;" ::"n"(LATER) : "memory");
}
// Tiles are asked for one ahead at d = 64 (2 x 4096 x 8 heads of 64, window 512: forward 342
// us, and 396 loaded in place).  At d = 128 the second buffer would cost the second CTA of
// an SM.
constexpr int tiles_ahead(int d) { return d == 64 ? 1 : 0; }

// s[i][j] += A[ra + i] . B[cb + 16 j] over D.
template <int D, int NI, int NJ>
__device__ __forceinline__ void dot_tile(float (&s)[NI][NJ], const float *A, int ra, const float *B, int cb)
{
#pragma unroll 4
    for (int x = 0; x < D; x += 4) {
        float4 u[NI], w[NJ];
#pragma unroll
        for (int i = 0; i < NI; ++i) u[i] = *reinterpret_cast<const float4 *>(A + (ra + i) * (D + 4) + x);
#pragma unroll
        for (int j = 0; j < NJ; ++j) w[j] = *reinterpret_cast<const float4 *>(B + (cb + 16 * j) * (D + 4) + x);
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                s[i][j] = fmaf(u[i].x, w[j].x, fmaf(u[i].y, w[j].y, fmaf(u[i].z, w[j].z, fmaf(u[i].w, w[j].w, s[i][j]))));
    }
}

// acc[i][c] += sum_j P[ra + i][j] V[j][cols of tx], NK rows of V, P with row stride PS.
template <int D, int NK, int PS>
__device__ __forceinline__ void mul_tile(float (&acc)[4][D / 16], const float *P, int ra, const float *V, int tx)
{
#pragma unroll 2
    for (int j = 0; j < NK; j += 4) {
        float4 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4 *>(P + (ra + i) * PS + j);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const float4 v = *reinterpret_cast<const float4 *>(V + (j + r) * (D + 4) + tx * 4 + 64 * c);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float w = r == 0 ? p[i].x : r == 1 ? p[i].y : r == 2 ? p[i].z : p[i].w;
                    acc[i][4 * c] = fmaf(w, v.x, acc[i][4 * c]);
                    acc[i][4 * c + 1] = fmaf(w, v.y, acc[i][4 * c + 1]);
                    acc[i][4 * c + 2] = fmaf(w, v.z, acc[i][4 * c + 2]);
                    acc[i][4 * c + 3] = fmaf(w, v.w, acc[i][4 * c + 3]);
                }
            }
    }
}

// acc[i][c] += sum_r P[r][ka + i] Q[r][cols of tx], NR rows, P with row stride PS.
template <int D, int NR, int PS>
__device__ __forceinline__ void mul_tile_t(float (&acc)[4][D / 16], const float *P, int ka, const float *Q, int tx)
{
#pragma unroll 4
    for (int r = 0; r < NR; ++r) {
        const float4 p = *reinterpret_cast<const float4 *>(P + r * PS + ka);
        const float w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            const float4 v = *reinterpret_cast<const float4 *>(Q + r * (D + 4) + tx * 4 + 64 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[i][4 * c] = fmaf(w[i], v.x, acc[i][4 * c]);
                acc[i][4 * c + 1] = fmaf(w[i], v.y, acc[i][4 * c + 1]);
                acc[i][4 * c + 2] = fmaf(w[i], v.z, acc[i][4 * c + 2]);
                acc[i][4 * c + 3] = fmaf(w[i], v.w, acc[i][4 * c + 3]);
            }
        }
    }
}

__device__ __forceinline__ float max16(float x)
{
#pragma unroll
    for (int o = 8; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, o));
    return x;
}
__device__ __forceinline__ float sum16(float x)
{
#pragma unroll
    for (int o = 8; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    return x;
}

// Writes row `t` (columns of tx) scaled by f; true if any of them is not finite.
template <typename E, int D>
__device__ __forceinline__ bool store_cols(E *dst, const float (&acc)[D / 16], float f, int tx)
{
    bool bad = false;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
        const float4 v = make_float4(acc[4 * c] * f, acc[4 * c + 1] * f, acc[4 * c + 2] * f, acc[4 * c + 3] * f);
        bad |= !(isfinite(v.x) && isfinite(v.y) && isfinite(v.z) && isfinite(v.w));
        store4(dst + tx * 4 + 64 * c, v);
    }
    return bad;
}

template <typename E, int D>
__global__ void __launch_bounds__(kThreads) fwd_kernel(const SwaArgs a)
{
    constexpr int LD = D + 4, PS = 68, AHEAD = tiles_ahead(D);
    extern __shared__ float sm[];
    float *Qs = sm, *Ks = Qs + 64 * LD, *Vs = Ks + AHEAD * 64 * LD, *Ps = Vs + 64 * LD;  // (one after the other in one place, or each its own)
    __shared__ unsigned bad[2];
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int i0 = (gridDim.x - 1 - blockIdx.x) * 64, h = blockIdx.y, b = blockIdx.z;  // longest rows first
    const int n = seq_len(a, b), off = a.Tk - a.T, hk = h / (a.Hq / a.Hk);
    const Rows<E> q = rows_of<E>(a.q, a.qs, b, h), k = rows_of<E>(a.k, a.ks, b, hk), v = rows_of<E>(a.v, a.vs, b, hk);
    E *out = const_cast<E *>(dense_rows<E>(a.out, b, h, a.T, a.Hq, D)[0]);
    const long long ost = (long long)a.Hq * D, lrow = ((long long)b * a.Hq + h) * a.T;
    if (tid < 2) bad[tid] = 0;
    float o[4][D / 16] = {}, m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = -INFINITY, l[i] = 0.f;
    if (i0 < n) {
        load_rows<E, D, 64>(Qs, q, i0, n);
        const int p0 = off + i0, p1 = off + min(i0 + 64, n) - 1;
        const KeyTiles kt(p0, p1, a.window, a.sinks, 64);
        const int keys = off + n;  // behind them is padding: zeros in the tile
        if (AHEAD) ask_rows<E, D, 64>(Ks, k, kt.tile(0) * 64, keys);
        rows_asked();
        for (int c = 0; c < kt.count(); ++c) {
            const int j0 = kt.tile(c) * 64;
            __syncthreads();
            if (AHEAD) ask_rows<E, D, 64>(Vs, v, j0, keys);
            else ask_rows<E, D, 64>(Ks, k, j0, keys);
            rows_asked();
            rows_landed<AHEAD>();
            __syncthreads();
            float s[4][4] = {};
            dot_tile<D, 4, 4>(s, Qs, ty * 4, Ks, tx);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = sees(p0 + ty * 4 + i, j0 + tx + 16 * j, a.window, a.sinks) ? s[i][j] * (a.scale * kLog2E)
                                                                                        : -INFINITY;
                    mx = fmaxf(mx, s[i][j]);
                }
                const float mn = fmaxf(m[i], max16(mx)), ms = mn == -INFINITY ? 0.f : mn;
                const float f = exp2f(m[i] - ms);
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float e = exp2f(s[i][j] - ms);
                    sum += e;
                    Ps[(ty * 4 + i) * PS + tx + 16 * j] = e;
                }
                m[i] = mn;
                l[i] = l[i] * f + sum16(sum);
#pragma unroll
                for (int u = 0; u < D / 16; ++u) o[i][u] *= f;
            }
            __syncthreads();
            if (!AHEAD) ask_rows<E, D, 64>(Vs, v, j0, keys);
            else if (c + 1 < kt.count()) ask_rows<E, D, 64>(Ks, k, kt.tile(c + 1) * 64, keys);
            rows_asked();
            rows_landed<AHEAD>();
            __syncthreads();
            mul_tile<D, 64, PS>(o, Ps, ty * 4, Vs, tx);
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = i0 + ty * 4 + i;
        if (t >= a.T) continue;
        const bool live = t < n;
        if (!live)
#pragma unroll
            for (int u = 0; u < D / 16; ++u) o[i][u] = 0.f;
        const float inv = !live || l[i] == 0.f ? 0.f : 1.f / l[i];
        const bool nf = store_cols<E, D>(out + t * ost, o[i], inv, tx);
        if (live && nf) atomicOr(&bad[(ty * 4 + i) >> 5], 1u << ((ty * 4 + i) & 31));
        if (a.lse && tx == 0) a.lse[lrow + t] = !live || l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
    }
    __syncthreads();
    for (int r = tid >> 5; r < 64; r += kThreads / 32)
        if (bad[r >> 5] >> (r & 31) & 1) row_forward<E, D>(a, b, h, i0 + r);
}

// dq of 64 query rows, key tiles of 32.
template <typename E, int D>
__global__ void __launch_bounds__(kThreads) dq_kernel(const SwaArgs a)
{
    constexpr int LD = D + 4, PS = 36, AHEAD = tiles_ahead(D);
    extern __shared__ float sm[];
    float *Qs = sm, *Gs = Qs + 64 * LD, *tiles = Gs + 64 * LD, *Ps = tiles + (1 + AHEAD) * 64 * LD;  // tiles: K, V
    __shared__ unsigned bad[2];
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int i0 = (gridDim.x - 1 - blockIdx.x) * 64, h = blockIdx.y, b = blockIdx.z;
    const int n = seq_len(a, b), off = a.Tk - a.T, hk = h / (a.Hq / a.Hk);
    const Rows<E> q = rows_of<E>(a.q, a.qs, b, h), k = rows_of<E>(a.k, a.ks, b, hk), v = rows_of<E>(a.v, a.vs, b, hk);
    const Rows<E> g = dense_rows<E>(a.dO, b, h, a.T, a.Hq, D);
    E *out = const_cast<E *>(dense_rows<E>(a.dq, b, h, a.T, a.Hq, D)[0]);
    const long long ost = (long long)a.Hq * D, lrow = ((long long)b * a.Hq + h) * a.T;
    if (tid < 2) bad[tid] = 0;
    float acc[4][D / 16] = {}, lse[4], delta[4];
    if (i0 < n) {
        load_rows<E, D, 64>(Qs, q, i0, n);
        load_rows<E, D, 64>(Gs, g, i0, n);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = min(i0 + ty * 4 + i, n - 1);
            lse[i] = a.lse[lrow + t];
            delta[i] = a.delta[lrow + t];
        }
        const int p0 = off + i0, p1 = off + min(i0 + 64, n) - 1;
        const KeyTiles kt(p0, p1, a.window, a.sinks, 32);
        auto ask = [&](int c) {
            if (c < kt.count()) {
                float *to = tiles + (AHEAD ? c & 1 : 0) * 64 * LD;
                ask_rows<E, D, 32>(to, k, kt.tile(c) * 32, off + n);  // (padding arrives as zeros)
                ask_rows<E, D, 32>(to + 32 * LD, v, kt.tile(c) * 32, off + n);
            }
            rows_asked();
        };
        if (AHEAD) ask(0);
        for (int c = 0; c < kt.count(); ++c) {
            const int j0 = kt.tile(c) * 32;
            const float *Ks = tiles + (AHEAD ? c & 1 : 0) * 64 * LD, *Vs = Ks + 32 * LD;
            __syncthreads();
            ask(c + AHEAD);
            rows_landed<AHEAD>();
            __syncthreads();
            float s[4][2] = {}, dp[4][2] = {};
            dot_tile<D, 4, 2>(s, Qs, ty * 4, Ks, tx);
            dot_tile<D, 4, 2>(dp, Gs, ty * 4, Vs, tx);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const bool on = sees(p0 + ty * 4 + i, j0 + tx + 16 * j, a.window, a.sinks);
                    Ps[(ty * 4 + i) * PS + tx + 16 * j] =
                        on ? prob(s[i][j], a.scale * kLog2E, lse[i]) * (dp[i][j] - delta[i]) : 0.f;
                }
            __syncthreads();
            mul_tile<D, 32, PS>(acc, Ps, ty * 4, Ks, tx);
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = i0 + ty * 4 + i;
        if (t >= a.T) continue;
        if (t >= n)
#pragma unroll
            for (int u = 0; u < D / 16; ++u) acc[i][u] = 0.f;
        if (store_cols<E, D>(out + t * ost, acc[i], a.scale, tx)) atomicOr(&bad[(ty * 4 + i) >> 5], 1u << ((ty * 4 + i) & 31));
    }
    __syncthreads();
    for (int r = tid >> 5; r < 64; r += kThreads / 32)
        if (bad[r >> 5] >> (r & 31) & 1) row_dq<E, D>(a, b, h, i0 + r);
}

// dk and dv of 64 keys, query tiles of 32 rows over all heads of the group.  With nsplit
// > 1 the (head, query tile) pairs of a key tile are dealt to nsplit CTAs, whose sums
// another kernel adds in order: part [nsplit][B][Hk][Tk][2][D].
template <typename E, int D>
__global__ void __launch_bounds__(kThreads) dkdv_kernel(const SwaArgs a, int nsplit, float *part)
{
    constexpr int LD = D + 4, PS = 68, AHEAD = tiles_ahead(D);
    extern __shared__ float sm[];
    float *Ks = sm, *Vs = Ks + 64 * LD, *tiles = Vs + 64 * LD, *Ps = tiles + (1 + AHEAD) * 64 * LD;  // tiles: Q, dO
    __shared__ unsigned bad[2];
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int j0 = (int)(blockIdx.x / nsplit) * 64, split = blockIdx.x % nsplit, hk = blockIdx.y, b = blockIdx.z;
    const int n = seq_len(a, b), off = a.Tk - a.T, G = a.Hq / a.Hk;
    if (tid < 2) bad[tid] = 0;
    float dk[4][D / 16] = {}, dv[4][D / 16] = {};
    load_rows<E, D, 64>(Ks, rows_of<E>(a.k, a.ks, b, hk), j0, a.Tk);
    load_rows<E, D, 64>(Vs, rows_of<E>(a.v, a.vs, b, hk), j0, a.Tk);
    const int i_lo = max(j0 - off, 0);
    const long long far = (long long)min(j0 + 64, a.Tk) - 1 + a.window - off;  // first row behind every window
    const int i_hi = (j0 < a.sinks || far > n) ? n : (int)far;
    const int nq = i_hi > i_lo ? (i_hi - i_lo + 31) / 32 : 0;
    const long long all = (long long)G * nq, per = (all + nsplit - 1) / nsplit;
    const long long it0 = split * per, it1 = min(all, (split + 1) * per);
    auto ask = [&](long long it) {
        if (it < it1) {
            const int h = hk * G + (int)(it / nq), i0 = i_lo + (int)(it % nq) * 32;
            float *to = tiles + (AHEAD ? (it - it0) & 1 : 0) * 64 * LD;
            ask_rows<E, D, 32>(to, rows_of<E>(a.q, a.qs, b, h), i0, n);
            ask_rows<E, D, 32>(to + 32 * LD, dense_rows<E>(a.dO, b, h, a.T, a.Hq, D), i0, n);
        }
        rows_asked();
    };
    if (AHEAD) ask(it0);
    for (long long it = it0; it < it1; ++it) {
        const int h = hk * G + (int)(it / nq), i0 = i_lo + (int)(it % nq) * 32;
        const long long lrow = ((long long)b * a.Hq + h) * a.T;
        const float *Qs = tiles + (AHEAD ? (it - it0) & 1 : 0) * 64 * LD, *Gs = Qs + 32 * LD;
        {
            __syncthreads();
            ask(it + AHEAD);
            rows_landed<AHEAD>();
            __syncthreads();
            float s[2][4] = {}, dp[2][4] = {};
            dot_tile<D, 2, 4>(s, Qs, ty * 2, Ks, tx);
            dot_tile<D, 2, 4>(dp, Gs, ty * 2, Vs, tx);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = i0 + ty * 2 + i, tc = min(t, n - 1);
                const float lse = a.lse[lrow + tc], delta = a.delta[lrow + tc];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool on = t < n && sees(off + t, j0 + tx + 16 * j, a.window, a.sinks);
                    s[i][j] = on ? prob(s[i][j], a.scale * kLog2E, lse) : 0.f;
                    dp[i][j] = on ? s[i][j] * (dp[i][j] - delta) : 0.f;
                    Ps[(ty * 2 + i) * PS + tx + 16 * j] = s[i][j];
                }
            }
            __syncthreads();
            mul_tile_t<D, 32, PS>(dv, Ps, ty * 4, Gs, tx);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) Ps[(ty * 2 + i) * PS + tx + 16 * j] = dp[i][j];
            __syncthreads();
            mul_tile_t<D, 32, PS>(dk, Ps, ty * 4, Qs, tx);
        }
    }
    __syncthreads();
    if (nsplit > 1) {
        float *out = part + ((((long long)split * a.B + b) * a.Hk + hk) * a.Tk) * 2 * D;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = j0 + ty * 4 + i;
            if (j >= a.Tk) continue;
            store_cols<float, D>(out + (long long)j * 2 * D, dk[i], a.scale, tx);
            store_cols<float, D>(out + (long long)j * 2 * D + D, dv[i], 1.f, tx);
        }
        return;
    }
    E *ok = const_cast<E *>(dense_rows<E>(a.dk, b, hk, a.Tk, a.Hk, D)[0]);
    E *ov = const_cast<E *>(dense_rows<E>(a.dv, b, hk, a.Tk, a.Hk, D)[0]);
    const long long st = (long long)a.Hk * D;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = j0 + ty * 4 + i;
        if (j >= a.Tk) continue;
        bool nf = store_cols<E, D>(ok + j * st, dk[i], a.scale, tx);
        nf |= store_cols<E, D>(ov + j * st, dv[i], 1.f, tx);
        if (nf) atomicOr(&bad[(ty * 4 + i) >> 5], 1u << ((ty * 4 + i) & 31));
    }
    __syncthreads();
    for (int r = tid >> 5; r < 64; r += kThreads / 32)
        if (bad[r >> 5] >> (r & 31) & 1) row_dkdv<E, D>(a, b, hk, j0 + r);
}

// The segments' sums added in order, one warp a key.
template <typename E, int D>
__global__ void __launch_bounds__(kThreads) dkdv_sum_kernel(const SwaArgs a, int nsplit, const float *part)
{
    const long long row = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), rows = (long long)a.B * a.Hk * a.Tk;
    if (row >= rows) return;  // row = (b, hk, j)
    const int lane = threadIdx.x & 31, j = (int)(row % a.Tk), hk = (int)(row / a.Tk % a.Hk), b = (int)(row / a.Tk / a.Hk);
    float v[2 * D / 32] = {};
    for (int s = 0; s < nsplit; ++s)
#pragma unroll
        for (int u = 0; u < 2 * D / 32; ++u) v[u] += part[(s * rows + row) * 2 * D + lane + 32 * u];
    const long long at = (((long long)b * a.Tk + j) * a.Hk + hk) * D;
    bool bad = false;
#pragma unroll
    for (int u = 0; u < D / 32; ++u) {
        bad |= !isfinite(v[u]) || !isfinite(v[D / 32 + u]);
        static_cast<E *>(a.dk)[at + lane + 32 * u] = from_f32<E>(v[u]);
        static_cast<E *>(a.dv)[at + lane + 32 * u] = from_f32<E>(v[D / 32 + u]);
    }
    if (__any_sync(~0u, bad)) row_dkdv<E, D>(a, b, hk, j);
}

// How many CTAs share a key tile: as many as bring the grid to twice the SMs, while each
// keeps four query tiles or more.
int kv_split(const SwaArgs &a, int num_sms)
{
    const long long ctas = (long long)((a.Tk + 63) / 64) * a.Hk * a.B;
    const long long seen = a.sinks > 0 ? a.T : (a.window + 63LL < a.T ? a.window + 63LL : a.T);
    const long long tiles = (seen + 31) / 32 * (a.Hq / a.Hk);
    int n = 1;
    while (n < 8 && ctas * n < 2LL * num_sms && tiles / (n * 2) >= 4) n *= 2;
    return n;
}

// delta = dO . o of every row that holds a token (0 in the others), a sequence in grid y: 16
// bytes a lane, so 8 to 32 lanes a row, and kDeltaRows rows a lane.  Bound by HBM and the
// division behind a row's place (4 x 4096 x 16 heads of 128 bf16: 28 us; with four rows a
// lane and two divisions a row 45).
constexpr int kDeltaRows = 2;
__device__ __forceinline__ long long quotient(long long n, int d)  // (64-bit division takes as long as the loads)
{
    return n < 0x7fffffffLL ? (unsigned)n / (unsigned)d : n / d;
}
template <typename E, int D>
__global__ void __launch_bounds__(kThreads) delta_kernel(const SwaArgs a)
{
    constexpr int W = 16 / sizeof(E), LPR = D / W, RPC = kThreads / LPR;  // elements a lane, lanes a row, rows at a time
    const long long rows = (long long)a.T * a.Hq, row0 = (long long)blockIdx.x * (RPC * kDeltaRows) + threadIdx.x / LPR;
    const int x = threadIdx.x % LPR * W, b = blockIdx.y, n = seq_len(a, b);
    const E *o_seq = static_cast<const E *>(a.o) + b * rows * D, *g_seq = static_cast<const E *>(a.dO) + b * rows * D;
    uint4 o[kDeltaRows], g[kDeltaRows];
    bool live[kDeltaRows];
    long long to[kDeltaRows];
#pragma unroll
    for (int u = 0; u < kDeltaRows; ++u) {
        const long long row = row0 + u * RPC;  // (t, h)
        const int t = (int)quotient(row, a.Hq), h = (int)(row - (long long)t * a.Hq);
        live[u] = row < rows && t < n;
        to[u] = row < rows ? ((long long)b * a.Hq + h) * a.T + t : -1;
        o[u] = g[u] = make_uint4(0, 0, 0, 0);
        if (live[u]) {
            o[u] = *reinterpret_cast<const uint4 *>(o_seq + row * D + x);
            g[u] = *reinterpret_cast<const uint4 *>(g_seq + row * D + x);
        }
    }
#pragma unroll
    for (int u = 0; u < kDeltaRows; ++u) {
        const E *p = reinterpret_cast<const E *>(&o[u]), *r = reinterpret_cast<const E *>(&g[u]);
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < W; ++e) s = fmaf(to_f32(p[e]), to_f32(r[e]), s);
#pragma unroll
        for (int w = LPR / 2; w; w >>= 1) s += __shfl_xor_sync(~0u, s, w);
        if (x == 0 && to[u] >= 0) a.delta[to[u]] = live[u] ? s : 0.f;
    }
}

// The same from the probabilities, delta_i = sum_j P_ij (dO_i . v_j), for bf16 rows that see
// few keys: there dO . o carries the roundings of o and of the forward's P undiminished into
// every dS of the row (relative error of dq 2.9e-3 with 4 visible keys, 2.5e-3 with 8, 2.2e-3
// with 16, the outputs' own rounding being 1.7e-3), and a row's scores are quickly formed
// again (4 x 4096 x 16 heads of 128, window 12: 509 us of backward, and 320 without).
// Short sequences see half of their keys on average.
constexpr int kFewKeys = 12;
template <int D>
__global__ void __launch_bounds__(kThreads) delta_few_kernel(const SwaArgs a)
{
    using E = __nv_bfloat16;
    constexpr int LPR = D / 8;
    const long long row = (long long)blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;  // (t, h)
    const bool in = row < (long long)a.T * a.Hq;
    const int b = blockIdx.y, t = in ? (int)quotient(row, a.Hq) : 0, h = in ? (int)(row - (long long)t * a.Hq) : 0;
    const bool live = in && t < seq_len(a, b);
    const int x = threadIdx.x % LPR * 8, hk = h / (a.Hq / a.Hk);
    const long long out = ((long long)b * a.Hq + h) * a.T + t;
    const Rows<E> k = rows_of<E>(a.k, a.ks, b, hk), v = rows_of<E>(a.v, a.vs, b, hk);
    const int p = a.Tk - a.T + t, lo = p - a.window + 1 > 0 ? p - a.window + 1 : 0;
    const int ns = a.sinks < lo ? a.sinks : lo, n = live ? ns + p + 1 - lo : 0;
    float q[8] = {}, g[8] = {}, lse = 0.f, sum = 0.f;
    auto dot = [](const float (&f)[8], uint4 u) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            s = fmaf(f[2 * e], __uint_as_float(w[e] << 16), fmaf(f[2 * e + 1], __uint_as_float(w[e] & 0xffff0000u), s));
        return s;
    };
    if (live) {
        const E *qr = rows_of<E>(a.q, a.qs, b, h)[t] + x, *gr = dense_rows<E>(a.dO, b, h, a.T, a.Hq, D)[t] + x;
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = to_f32(qr[e]), g[e] = to_f32(gr[e]);
        lse = a.lse[out];
    }
    const int most = __reduce_max_sync(~0u, n);  // (rows of a warp differ in length; all its lanes sum)
    for (int i0 = 0; i0 < most; i0 += 4) {       // four keys in flight
        uint4 kr[4], vr[4];
        float s[4], d[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u, j = i < ns ? i : lo + i - ns;
            kr[u] = vr[u] = make_uint4(0, 0, 0, 0);
            if (i < n) {
                kr[u] = *reinterpret_cast<const uint4 *>(k[j] + x);
                vr[u] = *reinterpret_cast<const uint4 *>(v[j] + x);
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) s[u] = dot(q, kr[u]), d[u] = dot(g, vr[u]);
#pragma unroll
        for (int w = LPR / 2; w; w >>= 1)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                s[u] += __shfl_xor_sync(~0u, s[u], w);
                d[u] += __shfl_xor_sync(~0u, d[u], w);
            }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (i0 + u < n) sum = fmaf(prob(s[u], a.scale * kLog2E, lse), d[u], sum);
    }
    if (x == 0 && in) a.delta[out] = live ? sum : 0.f;
}

template <typename E, int D>
cudaError_t fwd_impl(const SwaArgs &a, cudaStream_t stream)
{
    constexpr int bytes = sizeof(float) * ((2 + tiles_ahead(D)) * 64 * (D + 4) + 64 * 68);
    static std::atomic<unsigned long long> set{0};
    const cudaError_t e = ensure_smem_limit(fwd_kernel<E, D>, bytes, set);
    if (e != cudaSuccess) return e;
    return launch_plain(fwd_kernel<E, D>, dim3((a.T + 63) / 64, a.Hq, a.B), dim3(kThreads), bytes, stream, a);
}

template <typename E, int D>
cudaError_t bwd_impl(const SwaArgs &a, float *part, int num_sms, cudaStream_t stream)
{
    constexpr int rows = 192 + tiles_ahead(D) * 64, dq_bytes = sizeof(float) * (rows * (D + 4) + 64 * 36), kv_bytes = sizeof(float) * (rows * (D + 4) + 32 * 68);
    static std::atomic<unsigned long long> dq_set{0}, kv_set{0};
    cudaError_t e = ensure_smem_limit(dq_kernel<E, D>, dq_bytes, dq_set);
    if (e == cudaSuccess) e = ensure_smem_limit(dkdv_kernel<E, D>, kv_bytes, kv_set);
    if (e == cudaSuccess)
        e = launch_plain(dq_kernel<E, D>, dim3((a.T + 63) / 64, a.Hq, a.B), dim3(kThreads), dq_bytes, stream, a);
    const int nsplit = kv_split(a, num_sms);
    if (e == cudaSuccess)
        e = launch_plain(dkdv_kernel<E, D>, dim3((a.Tk + 63) / 64 * nsplit, a.Hk, a.B), dim3(kThreads), kv_bytes, stream, a, nsplit,
                         part);
    if (e != cudaSuccess || nsplit == 1) return e;
    const long long keys = (long long)a.B * a.Hk * a.Tk;
    return launch_plain(dkdv_sum_kernel<E, D>, dim3((unsigned)((keys + 7) / 8)), dim3(kThreads), 0, stream, a, nsplit,
                        (const float *)part);
}

template <typename E, int D>
cudaError_t delta_impl(const SwaArgs &a, cudaStream_t stream)
{
    const bool few = sizeof(E) == 2 && ((long long)a.window + a.sinks <= kFewKeys || a.Tk <= 2 * kFewKeys);
    const int per = kThreads * 16 / (D * (int)sizeof(E)) * (few ? 1 : kDeltaRows);
    const long long rows = (long long)a.T * a.Hq, blocks = (rows + per - 1) / per;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_plain(few ? delta_few_kernel<D> : delta_kernel<E, D>, dim3((unsigned)blocks, a.B), dim3(kThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_swa_fwd_simt(const SwaArgs &a, cudaStream_t stream)
{
    return a.d == 128 ? fwd_impl<float, 128>(a, stream) : fwd_impl<float, 64>(a, stream);
}

size_t swa_bwd_simt_partial_floats(const SwaArgs &a, int num_sms)
{
    const int n = kv_split(a, num_sms);
    return n > 1 ? (size_t)n * a.B * a.Hk * a.Tk * 2 * a.d : 0;
}

cudaError_t launch_swa_bwd_simt(const SwaArgs &a, float *part, int num_sms, cudaStream_t stream)
{
    return a.d == 128 ? bwd_impl<float, 128>(a, part, num_sms, stream) : bwd_impl<float, 64>(a, part, num_sms, stream);
}

cudaError_t launch_swa_delta(const SwaArgs &a, bool bf16, cudaStream_t stream)
{
    if (bf16) return a.d == 128 ? delta_impl<__nv_bfloat16, 128>(a, stream) : delta_impl<__nv_bfloat16, 64>(a, stream);
    return a.d == 128 ? delta_impl<float, 128>(a, stream) : delta_impl<float, 64>(a, stream);
}

}  // namespace gdn2
