// swa_decode.cu -- one token of the windowed attention against a ring cache.
//
// A cluster of CTAs shares one (batch, key/value head): each CTA takes a run of the
// visible positions, each of its warps every fourth group of them, and the partial (max,
// sum, output) triples are joined through shared memory, then through distributed shared
// memory -- one launch, no workspace.  Bound by HBM: the visible cache is read once for
// all query heads of the group.
//
// bf16: warp-level matrix instructions over 16 heads x 16 keys.  Keys and values go from
// memory straight into operand registers, 16 bytes a load: a dot product does not care in
// which order its channels are taken, so a lane's 16 bytes of a key serve as two k-steps
// of it (the query is loaded in the same order), and an output tile takes every eighth
// channel so that a lane's 16 bytes of a value row feed eight tiles.  (The fifth-generation
// tensor core would need the rows in shared memory first; a step of 16 keys is 64 warp
// instructions here against 8 KB from memory, so it would not be used a tenth.)
// fp32: one key row per half or whole warp on the CUDA cores.
#include <cooperative_groups.h>

#include "launch.h"
#include "swa_common.cuh"

namespace gdn2 {
namespace {

using namespace swa;
namespace cg = cooperative_groups;


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

// The warps' partial results of a CTA, and the CTA's.
template <int NW, int GC, int D>
struct Partials {
    float m[NW][GC], l[NW][GC];
    alignas(16) float o[NW][GC][D];
};
// What the CTAs of a cluster send to the one that joins a head: slot (CTA, head).
constexpr int kMaxSplit = 8;
template <int GC, int D>
struct Joined {
    static constexpr int HEADS = (GC + 1) / 2;  // of one joining CTA, when there are two or more
    float m[kMaxSplit][HEADS], l[kMaxSplit][HEADS], o[kMaxSplit][HEADS][D];
};

// A barrier of the cluster in two halves: every CTA has started (arrived) before another
// stores into its shared memory (waited), without holding up the work between.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

template <int NW, int GC, int D>
struct DecodeShared {
    Partials<NW, GC, D> part;
    Joined<GC, D> joined;
};

// Joins the warps, then the CTAs of the cluster, and writes the heads [0, ng).  Head g is
// joined by CTA g % nsplit: the others store their part into its shared memory (one way,
// where reading would be a round trip per value).
template <typename E, int D, int NW, int GC>
__device__ __forceinline__ void join(const Partials<NW, GC, D> &part, Joined<GC, D> &mine, E *out, int split, int nsplit, int ng)
{
    cg::cluster_group cluster = cg::this_cluster();
    __syncthreads();
    cluster_wait();
    for (int i = threadIdx.x; i < ng * D; i += blockDim.x) {
        const int g = i / D, d = i % D;
        float mn = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) mn = fmaxf(mn, part.m[w][g]);
        const float ms = mn == -INFINITY ? 0.f : mn;
        float sl = 0.f, so = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float f = exp2f(part.m[w][g] - ms);
            sl = fmaf(part.l[w][g], f, sl);
            so = fmaf(part.o[w][g][d], f, so);
        }
        if (nsplit == 1) {
            out[g * D + d] = from_f32<E>(sl == 0.f ? 0.f : so / sl);
        } else {
            const int to = g % nsplit, at = g / nsplit;
            *cluster.map_shared_rank(&mine.o[split][at][d], to) = so;
            if (d == 0) {
                *cluster.map_shared_rank(&mine.m[split][at], to) = mn;
                *cluster.map_shared_rank(&mine.l[split][at], to) = sl;
            }
        }
    }
    if (nsplit == 1) return;
    cluster.sync();
    for (int i = threadIdx.x; i < ng * D; i += blockDim.x) {
        const int at = i / D, d = i % D, g = at * nsplit + split;
        if (g >= ng) break;
        float mn = -INFINITY;
        for (int r = 0; r < nsplit; ++r) mn = fmaxf(mn, mine.m[r][at]);
        const float ms = mn == -INFINITY ? 0.f : mn;
        float sl = 0.f, so = 0.f;
        for (int r = 0; r < nsplit; ++r) {
            const float f = exp2f(mine.m[r][at] - ms);
            sl = fmaf(mine.l[r][at], f, sl);
            so = fmaf(mine.o[r][at][d], f, so);
        }
        out[g * D + d] = from_f32<E>(sl == 0.f ? 0.f : so / sl);
    }
}

// GC query heads of the group per CTA; lanes hold 4 channels each of D / 4 lanes per key.
template <typename E, int D, int GC>
__global__ void __launch_bounds__(4 * 32) decode_kernel(const SwaDecodeArgs a, int nsplit, int nchunk)
{
    constexpr int LPR = D / 4, KPW = 32 / LPR;  // lanes per key, keys per warp step
    constexpr int U = 4, NW = 4;                // steps in flight, warps
    using Shared = DecodeShared<NW, GC, D>;
    extern __shared__ __align__(16) uint8_t dyn[];
    auto &part = reinterpret_cast<Shared *>(dyn)->part;
    auto &joined = reinterpret_cast<Shared *>(dyn)->joined;
    const int split = blockIdx.x, hk = blockIdx.y / nchunk, chunk = blockIdx.y % nchunk, b = blockIdx.z;
    const int G = a.Hq / a.Hk, g0 = chunk * GC, ng = min(GC, G - g0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / LPR, x = lane % LPR * 4;
    E *out = static_cast<E *>(a.o) + ((long long)b * a.Hq + hk * G + g0) * D;
    cluster_arrive();
    const int P = a.pos[b];
    if (P < 0) {  // no sequence in this row
        cluster_wait();
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
    for (int t = t0 + warp * KPW * U; t < t1; t += NW * KPW * U) {
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
    // the keys of a warp's sub-rows
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
            for (int c = 0; c < 4; ++c) part.o[warp][g][x + c] = o[g][c];
            if (lane == 0) part.m[warp][g] = m[g], part.l[warp][g] = l[g];
        }
    }
    join<E, D, NW, GC>(part, joined, out, split, nsplit, ng);
}

// One step of 16 heads x 8 keys (or 8 channels): D += A B, bf16 operands.
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with heads 8..15 absent: their half of the result is not kept.
__device__ __forceinline__ void mma_bf16(float (&d)[2], uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1)
{
    [[maybe_unused]] float none0, none1;
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%5}, {%7,%8}, {%0,%1,%9,%9};"
                 : "+f"(d[0]), "+f"(d[1]), "=f"(none0), "=f"(none1)
                 : "r"(a0), "r"(0), "r"(a2), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t pair_bf16(float x, float y)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint4 load_stream(const __nv_bfloat16 *p)
{
    uint4 v;  // (not through the read-only path: another CTA of the cluster may just have put the new token there)
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// HR x 8 query heads of a CTA: both halves of the matrix instruction's rows, or one (whose
// registers then let a third CTA onto the SM, and more loads into flight).
template <int D, int HR, int NW>
__global__ void __launch_bounds__(NW * 32, NW == 8 ? 1 : HR == 1 && D == 64 ? 4 : 2) decode_mma_kernel(const SwaDecodeArgs a, int nsplit, int nchunk)
{
    using E = __nv_bfloat16;
    constexpr int kHeads = 8 * HR;
    constexpr int NC = D / 32;  // 16-byte chunks of a row per lane
    using Shared = DecodeShared<NW, kHeads, D>;
    extern __shared__ __align__(16) uint8_t dyn[];
    auto &part = reinterpret_cast<Shared *>(dyn)->part;
    auto &joined = reinterpret_cast<Shared *>(dyn)->joined;
    const int split = blockIdx.x, hk = blockIdx.y / nchunk, chunk = blockIdx.y % nchunk, b = blockIdx.z;
    const int G = a.Hq / a.Hk, g0 = chunk * kHeads, ng = min(kHeads, G - g0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, c = lane & 3;
    E *out = static_cast<E *>(a.o) + ((long long)b * a.Hq + hk * G + g0) * D;
    cluster_arrive();
    const int P = a.pos[b];
    if (P < 0) {  // no sequence in this row
        cluster_wait();
        if (split == 0)
            for (int i = threadIdx.x; i < ng * D; i += blockDim.x) out[i] = from_f32<E>(0.f);
        return;
    }
    const E *kn = static_cast<const E *>(a.k) + b * a.ks[0] + hk * a.ks[1];
    const E *vn = static_cast<const E *>(a.v) + b * a.vs[0] + hk * a.vs[1];
    if (split == 0 && chunk == 0) put_new_token<E>(a, b, hk, P, kn, vn);
    const Visible vis(P, a.window, a.sinks, a.slots);
    const long long cache0 = ((long long)b * a.slots * a.Hk + hk) * D, cstep = (long long)a.Hk * D;
    const E *kc = static_cast<const E *>(a.kc) + cache0, *vc = static_cast<const E *>(a.vc) + cache0;

    // query heads gr (and gr + 8), absent heads as zeros
    uint4 q[HR][NC];
#pragma unroll
    for (int r = 0; r < HR; ++r)
#pragma unroll
        for (int j = 0; j < NC; ++j)
            q[r][j] = gr + 8 * r < ng
                          ? *reinterpret_cast<const uint4 *>(static_cast<const E *>(a.q) + b * a.qs[0] +
                                                             (long long)(hk * G + g0 + gr + 8 * r) * a.qs[1] + (j * 4 + c) * 8)
                          : make_uint4(0, 0, 0, 0);

    const int per = (vis.n + nsplit - 1) / nsplit;
    const int t0 = split * per, t1 = min(vis.n, t0 + per);
    // rows behind the run read its last position again; their scores are masked
    auto row = [&](const E *fresh, const E *cache, int t) {
        const int p = vis.position(t < t1 ? t : t1 - 1);
        return p == P ? fresh : cache + vis.slot(p) * cstep;
    };
    uint4 kf[2][NC], vf[4][D / 64];
    auto load_keys = [&](int t) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const E *p = row(kn, kc, t + gr + 8 * r) + c * 8;
#pragma unroll
            for (int j = 0; j < NC; ++j) kf[r][j] = load_stream(p + j * 32);
        }
    };
    auto load_values = [&](int t) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const E *p = row(vn, vc, t + 2 * c + (r & 1) + (r >> 1) * 8) + gr * 8;
#pragma unroll
            for (int j = 0; j < D / 64; ++j) vf[r][j] = load_stream(p + j * 64);
        }
    };
    float m[HR], l[HR] = {}, o[D / 8][2 * HR] = {};
#pragma unroll
    for (int h = 0; h < HR; ++h) m[h] = -INFINITY;
    const float sc = a.scale * kLog2E;
    int t = t0 + warp * 16;
    if (t < t1) {
        load_keys(t);
        load_values(t);
    }
    for (; t < t1; t += NW * 16) {
        float s[2][2 * HR] = {};
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                if constexpr (HR == 2) {
                    mma_bf16(s[r], q[0][j].x, q[1][j].x, q[0][j].y, q[1][j].y, kf[r][j].x, kf[r][j].y);
                    mma_bf16(s[r], q[0][j].z, q[1][j].z, q[0][j].w, q[1][j].w, kf[r][j].z, kf[r][j].w);
                } else {
                    mma_bf16(s[r], q[0][j].x, q[0][j].y, kf[r][j].x, kf[r][j].y);
                    mma_bf16(s[r], q[0][j].z, q[0][j].w, kf[r][j].z, kf[r][j].w);
                }
            }
        const int tn = t + NW * 16;
        if (tn < t1) load_keys(tn);
        // s[r][0..1]: head gr, keys 8 r + 2 c + {0, 1}; s[r][2..3]: head gr + 8
        float mx[HR];
        bool grow = false;
#pragma unroll
        for (int h = 0; h < HR; ++h) {
            mx[h] = -INFINITY;
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float &v = s[r][2 * h + e];
                    v = t + 8 * r + 2 * c + e < t1 ? v * sc : -INFINITY;
                    mx[h] = fmaxf(mx[h], v);
                }
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(~0u, mx[h], 1));
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(~0u, mx[h], 2));
            grow |= mx[h] > m[h] + 8.f;
        }
        // the reference of a head is raised only when it is outgrown by more than 2^8
        if (__any_sync(~0u, grow)) {
#pragma unroll
            for (int h = 0; h < HR; ++h) {
                const bool up = mx[h] > m[h] + 8.f;
                const float f = up ? exp2f(m[h] - mx[h]) : 1.f;
                if (up) m[h] = mx[h];
                l[h] *= f;
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    o[n][2 * h] *= f;
                    o[n][2 * h + 1] *= f;
                }
            }
        }
#pragma unroll
        for (int h = 0; h < HR; ++h) {
            const float ms = m[h] == -INFINITY ? 0.f : m[h];
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float &v = s[r][2 * h + e];
                    v = exp2f(v - ms);
                    l[h] += v;
                }
        }
        // P rounded to bf16 for the product (the sum keeps the unrounded values)
        uint32_t p[2][HR];  // [keys 0..7, 8..15][heads 0..7, 8..15]
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int h = 0; h < HR; ++h) p[r][h] = pair_bf16(s[r][2 * h], s[r][2 * h + 1]);
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            const uint32_t *w0 = &vf[0][j].x, *w1 = &vf[1][j].x, *w2 = &vf[2][j].x, *w3 = &vf[3][j].x;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                const uint32_t sel = n & 1 ? 0x7632 : 0x5410;
                const uint32_t b0 = __byte_perm(w0[n / 2], w1[n / 2], sel), b1 = __byte_perm(w2[n / 2], w3[n / 2], sel);
                if constexpr (HR == 2) mma_bf16(o[j * 8 + n], p[0][0], p[0][1], p[1][0], p[1][1], b0, b1);
                else mma_bf16(o[j * 8 + n], p[0][0], p[1][0], b0, b1);
            }
        }
        if (tn < t1) load_values(tn);
    }
    // o[j * 8 + n][0..1]: head gr, channels 64 j + 8 (2 c + {0, 1}) + n; [2..3]: head gr + 8
#pragma unroll
    for (int h = 0; h < HR; ++h) {
        l[h] += __shfl_xor_sync(~0u, l[h], 1);
        l[h] += __shfl_xor_sync(~0u, l[h], 2);
        const int head = gr + 8 * h;
        if (c == 0) part.m[warp][head] = m[h], part.l[warp][head] = l[h];
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int n = 0; n < 8; n += 4)
                    *reinterpret_cast<float4 *>(&part.o[warp][head][64 * j + 8 * (2 * c + e) + n]) =
                        make_float4(o[j * 8 + n][2 * h + e], o[j * 8 + n + 1][2 * h + e], o[j * 8 + n + 2][2 * h + e],
                                    o[j * 8 + n + 3][2 * h + e]);
    }
    join<E, D, NW, kHeads>(part, joined, out, split, nsplit, ng);
}

// CTAs that share a (sequence, heads) row: the number with the least waves x time of a
// CTA, whose own cost (query, join, cluster) counts as much as about 300 positions
// (64 x 4 rows of 2052 positions of 128 bf16: 103 us split in 8, 78 in 4, 68 in 2).
int splits(const SwaDecodeArgs &a, int gc, int per_sm, int num_sms)
{
    const int G = a.Hq / a.Hk, nchunk = (G + gc - 1) / gc;
    const long long rows = (long long)a.B * a.Hk * nchunk, seen = (long long)a.window + a.sinks, fit = (long long)per_sm * num_sms;
    int best = 1;
    double least = 0;
    for (int n = 1; n <= kMaxSplit; n *= 2) {
        const double cost = (double)((rows * n + fit - 1) / fit) * ((double)seen / n + 300.0);
        if (n == 1 || cost < least) least = cost, best = n;
    }
    return best;
}

// GC query heads of a group and NW warps per CTA, PER_SM CTAs on an SM.
template <auto kern, int GC, int D, int NW, int PER_SM>
cudaError_t launch(const SwaDecodeArgs &a, int num_sms, cudaStream_t stream)
{
    constexpr int gc = GC, bytes = sizeof(DecodeShared<NW, GC, D>);
    static std::atomic<unsigned long long> set{0};
    cudaError_t e = ensure_smem_limit(kern, bytes, set);
    if (e != cudaSuccess) return e;
    const int G = a.Hq / a.Hk, nchunk = (G + gc - 1) / gc, nsplit = splits(a, gc, PER_SM, num_sms);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(nsplit, a.Hk * nchunk, a.B);  // (y is at most the number of query heads)
    cfg.blockDim = dim3(NW * 32);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = nsplit;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = nsplit > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a, nsplit, nchunk);
}

template <int D>
cudaError_t by_group_f32(const SwaDecodeArgs &a, int num_sms, cudaStream_t stream)
{
    const int G = a.Hq / a.Hk;
    if (G == 1) return launch<decode_kernel<float, D, 1>, 1, D, 4, 4>(a, num_sms, stream);
    if (G == 2) return launch<decode_kernel<float, D, 2>, 2, D, 4, 4>(a, num_sms, stream);
    return launch<decode_kernel<float, D, 4>, 4, D, 4, 4>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_swa_decode(const SwaDecodeArgs &a, bool bf16, int num_sms, cudaStream_t stream)
{
    if (bf16) {
        // few rows: eight warps a CTA, so that a warp's walk is short (one sequence, 16 heads of
        // 128, 2052 slots: 13.8 us with four)
        const bool small_group = a.Hq / a.Hk <= 8;
        if (small_group && (long long)a.B * a.Hk * kMaxSplit <= num_sms)
            return a.d == 128 ? launch<decode_mma_kernel<128, 1, 8>, 8, 128, 8, 1>(a, num_sms, stream)
                              : launch<decode_mma_kernel<64, 1, 8>, 8, 64, 8, 1>(a, num_sms, stream);
        if (small_group && a.d == 64) return launch<decode_mma_kernel<64, 1, 4>, 8, 64, 4, 4>(a, num_sms, stream);
        return a.d == 128 ? launch<decode_mma_kernel<128, 2, 4>, 16, 128, 4, 2>(a, num_sms, stream)
                          : launch<decode_mma_kernel<64, 2, 4>, 16, 64, 4, 2>(a, num_sms, stream);
    }
    return a.d == 128 ? by_group_f32<128>(a, num_sms, stream) : by_group_f32<64>(a, num_sms, stream);
}

}  // namespace gdn2
