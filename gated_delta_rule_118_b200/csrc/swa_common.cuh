// swa_common.cuh -- what the windowed-attention kernels share: which keys a row
// sees, which tiles a tile visits, and single rows computed one key at a time.
//
// Query row i of a sequence stands at position p = Tk - T + i and sees key j iff
// j <= p and (p - j < window or j < sinks).  Rows at or behind the sequence's
// length are padding and see nothing.
//
// Masked places and non-finite values: the tile kernels select masked scores away
// before the exponential, but their second products still multiply a zero
// probability with whatever stands in a masked row of v (k, q, dO in the
// backward), and 0 * NaN or 0 * infinity is NaN.  Rows of padding are therefore zeros in
// shared memory (only the tile at a sequence's end has any).  Scrubbing the other tiles
// would cost shared-memory bandwidth on every call, so a kernel instead looks at the row
// it is about to write: if it is not finite, the row is computed again from memory by
// one of the functions below, which touch visible keys only (unless its own row holds a
// NaN, which reaches all of it).  That takes one warp a row and is slow; it is for tokens
// of a sequence that are not finite, and for bf16 values beyond 2^67 or so, which a
// probability of up to 2^60 (relative to the row's reference) can take to infinity.  A
// row that is NaN by its own visible inputs comes out NaN again.
#pragma once

#include "common.cuh"
#include "hybrid.h"

namespace gdn2 {
namespace swa {

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ int seq_len(const SwaArgs &a, int b)
{
    if (!a.lens) return a.T;
    const int n = a.lens[b];
    return n < 0 ? 0 : n > a.T ? a.T : n;
}

__device__ __forceinline__ bool sees(int p, int j, int window, int sinks)
{
    return j <= p && (p - j < window || j < sinks);
}

// Key tiles (of BN keys) that rows at positions [p0, p1] visit: tiles [0, nsink)
// for the sinks behind the window, then tiles [w0, w1).
struct KeyTiles {
    int nsink, w0, w1;
    __device__ __forceinline__ KeyTiles(int p0, int p1, int window, int sinks, int BN)
    {
        const int lo = p0 - window + 1 > 0 ? p0 - window + 1 : 0;
        w0 = lo / BN;
        w1 = p1 / BN + 1;
        const int s = (sinks + BN - 1) / BN;
        nsink = s < w0 ? s : w0;
    }
    __device__ __forceinline__ int count() const { return nsink + w1 - w0; }
    __device__ __forceinline__ int tile(int n) const { return n < nsink ? n : w0 + n - nsink; }
};

// Rows [first, 128) of a tile in shared memory (boxes of 128 rows x 64 bf16 with the 128-byte
// swizzle, which stays within a row) set to zero by one warp, for tensor-core reads that
// follow a barrier.  What stands in the padding behind a sequence is not to meet a zero
// probability: not being finite, it would make every row of its tile be formed again.
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t *tile, int first)
{
    for (int x = 0; x < D / 64; ++x)
        for (int c = first * 8 + (threadIdx.x & 31); c < 128 * 8; c += 32)
            *reinterpret_cast<uint4 *>(tile + x * 16384 + c * 16) = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
}

// Whether all of keys [j0, j1) are visible to all of positions [p0, p1].
__device__ __forceinline__ bool tile_full(int p0, int p1, int j0, int j1, int window, int sinks)
{
    return j1 - 1 <= p0 && (p1 - j0 < window || j1 <= sinks);
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    return x;
}
__device__ __forceinline__ float warp_max(float x)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, o));
    return x;
}

template <typename E, int D>
__device__ __forceinline__ float dot_rows(const E *x, const E *y)
{
    float s = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
        const float4 u = load4(x + c), w = load4(y + c);
        s = fmaf(u.x, w.x, fmaf(u.y, w.y, fmaf(u.z, w.z, fmaf(u.w, w.w, s))));
    }
    return s;
}

// Whether a row holds a NaN (the whole warp asks): what is formed from such a row is NaN
// throughout, and need not be formed again.
template <typename E, int D>
__device__ __forceinline__ bool has_nan(const E *row)
{
    bool bad = false;
#pragma unroll
    for (int u = 0; u < D / 32; ++u) {
        const float x = to_f32(row[(threadIdx.x & 31) + 32 * u]);
        bad |= x != x;
    }
    return __any_sync(~0u, bad);
}

// Element pointers of one (batch, head).
template <typename E>
struct Rows {
    const E *p;
    long long st;
    __device__ __forceinline__ const E *operator[](int t) const { return p + (long long)t * st; }
};
template <typename E>
__device__ __forceinline__ Rows<E> rows_of(const void *base, const long long (&st)[3], int b, int h)
{
    return {static_cast<const E *>(base) + (long long)b * st[0] + (long long)h * st[2], st[1]};
}
template <typename E>
__device__ __forceinline__ Rows<E> dense_rows(const void *base, int b, int h, int T, int H, int D)
{
    return {static_cast<const E *>(base) + ((long long)b * T * H + h) * D, (long long)H * D};
}

// Row i of the forward, by one warp: o and lse written.
template <typename E, int D>
__device__ __forceinline__ void row_forward(const SwaArgs &a, int b, int h, int i)
{
    const int lane = threadIdx.x & 31, p = a.Tk - a.T + i;
    const E *q = rows_of<E>(a.q, a.qs, b, h)[i];
    if (has_nan<E, D>(q)) return;
    const int hk = h / (a.Hq / a.Hk);
    const Rows<E> k = rows_of<E>(a.k, a.ks, b, hk), v = rows_of<E>(a.v, a.vs, b, hk);
    const int lo = p - a.window + 1 > 0 ? p - a.window + 1 : 0;
    const int ns = a.sinks < lo ? a.sinks : lo, n = ns + p + 1 - lo;
    float m = -INFINITY, l = 0.f, o[D / 32] = {};
    for (int c = 0; c < n; c += 32) {
        const int t = c + lane, j = t < ns ? t : lo + t - ns;
        const bool on = t < n;
        const float s = on ? dot_rows<E, D>(q, k[j]) * (a.scale * kLog2E) : -INFINITY;
        const float mn = fmaxf(m, warp_max(s)), ms = mn == -INFINITY ? 0.f : mn;
        const float f = exp2f(m - ms), e = on ? exp2f(s - ms) : 0.f;
        m = mn;
        l = l * f + warp_sum(e);
#pragma unroll
        for (int u = 0; u < D / 32; ++u) o[u] *= f;
        const int live = n - c < 32 ? n - c : 32;
        for (int r = 0; r < live; ++r) {
            const int tr = c + r, jr = tr < ns ? tr : lo + tr - ns;
            const float w = __shfl_sync(~0u, e, r);
#pragma unroll
            for (int u = 0; u < D / 32; ++u) o[u] = fmaf(w, to_f32(v[jr][lane + 32 * u]), o[u]);
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    E *out = const_cast<E *>(dense_rows<E>(a.out, b, h, a.T, a.Hq, D)[i]);
#pragma unroll
    for (int u = 0; u < D / 32; ++u) out[lane + 32 * u] = from_f32<E>(o[u] * inv);
    if (a.lse && lane == 0)
        a.lse[((long long)b * a.Hq + h) * a.T + i] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// exp(scale * s - lse) of a visible pair; 0 for a row without any finite score.
__device__ __forceinline__ float prob(float s, float scale_log2e, float lse)
{
    return lse == -INFINITY ? 0.f : exp2f(s * scale_log2e - lse * kLog2E);
}

// Row i of dq, by one warp.
template <typename E, int D>
__device__ __forceinline__ void row_dq(const SwaArgs &a, int b, int h, int i)
{
    const int lane = threadIdx.x & 31, p = a.Tk - a.T + i;
    const E *q = rows_of<E>(a.q, a.qs, b, h)[i];
    const E *g = dense_rows<E>(a.dO, b, h, a.T, a.Hq, D)[i];
    if (has_nan<E, D>(q) || has_nan<E, D>(g)) return;
    const int hk = h / (a.Hq / a.Hk);
    const Rows<E> k = rows_of<E>(a.k, a.ks, b, hk), v = rows_of<E>(a.v, a.vs, b, hk);
    const long long row = ((long long)b * a.Hq + h) * a.T + i;
    const float lse = a.lse[row], delta = a.delta[row];
    const int lo = p - a.window + 1 > 0 ? p - a.window + 1 : 0;
    const int ns = a.sinks < lo ? a.sinks : lo, n = ns + p + 1 - lo;
    float acc[D / 32] = {};
    for (int c = 0; c < n; c += 32) {
        const int t = c + lane, j = t < ns ? t : lo + t - ns;
        float ds = 0.f;
        if (t < n)
            ds = prob(dot_rows<E, D>(q, k[j]), a.scale * kLog2E, lse) * (dot_rows<E, D>(g, v[j]) - delta) * a.scale;
        const int live = n - c < 32 ? n - c : 32;
        for (int r = 0; r < live; ++r) {
            const int tr = c + r, jr = tr < ns ? tr : lo + tr - ns;
            const float w = __shfl_sync(~0u, ds, r);
#pragma unroll
            for (int u = 0; u < D / 32; ++u) acc[u] = fmaf(w, to_f32(k[jr][lane + 32 * u]), acc[u]);
        }
    }
    E *out = const_cast<E *>(dense_rows<E>(a.dq, b, h, a.T, a.Hq, D)[i]);
#pragma unroll
    for (int u = 0; u < D / 32; ++u) out[lane + 32 * u] = from_f32<E>(acc[u]);
}

// Row j of dk and dv, by one warp.
template <typename E, int D>
__device__ __forceinline__ void row_dkdv(const SwaArgs &a, int b, int hk, int j)
{
    const int lane = threadIdx.x & 31, off = a.Tk - a.T, G = a.Hq / a.Hk;
    const E *k = rows_of<E>(a.k, a.ks, b, hk)[j], *v = rows_of<E>(a.v, a.vs, b, hk)[j];
    const int len = seq_len(a, b);
    const int i0 = j > off ? j - off : 0;
    const long long far = (long long)j + a.window - off;  // first row that no longer sees j through the window
    const int i1 = (j < a.sinks || far > len) ? len : (int)far;
    if (i0 < i1 && has_nan<E, D>(k)) return;
    float dk[D / 32] = {}, dv[D / 32] = {};
    for (int h = hk * G; h < hk * G + G; ++h) {
        const Rows<E> q = rows_of<E>(a.q, a.qs, b, h), g = dense_rows<E>(a.dO, b, h, a.T, a.Hq, D);
        const long long row = ((long long)b * a.Hq + h) * a.T;
        for (int c = i0; c < i1; c += 32) {
            const int i = c + lane;
            float pr = 0.f, ds = 0.f;
            if (i < i1) {
                pr = prob(dot_rows<E, D>(q[i], k), a.scale * kLog2E, a.lse[row + i]);
                ds = pr * (dot_rows<E, D>(g[i], v) - a.delta[row + i]) * a.scale;
            }
            const int live = i1 - c < 32 ? i1 - c : 32;
            for (int r = 0; r < live; ++r) {
                const float wp = __shfl_sync(~0u, pr, r), ws = __shfl_sync(~0u, ds, r);
#pragma unroll
                for (int u = 0; u < D / 32; ++u) {
                    dv[u] = fmaf(wp, to_f32(g[c + r][lane + 32 * u]), dv[u]);
                    dk[u] = fmaf(ws, to_f32(q[c + r][lane + 32 * u]), dk[u]);
                }
            }
        }
    }
    E *ok = const_cast<E *>(dense_rows<E>(a.dk, b, hk, a.Tk, a.Hk, D)[j]);
    E *ov = const_cast<E *>(dense_rows<E>(a.dv, b, hk, a.Tk, a.Hk, D)[j]);
#pragma unroll
    for (int u = 0; u < D / 32; ++u) {
        ok[lane + 32 * u] = from_f32<E>(dk[u]);
        ov[lane + 32 * u] = from_f32<E>(dv[u]);
    }
}

}  // namespace swa
}  // namespace gdn2
