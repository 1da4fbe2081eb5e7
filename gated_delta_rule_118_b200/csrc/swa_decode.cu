// swa_decode.cu -- one token of the windowed attention against a ring cache.
//
// A cluster of CTAs shares one (batch, key/value head): each CTA takes a run of the
// visible positions, each of its warps every fourth group of them, and the partial (max,
// sum, output) triples are joined through shared memory, then through distributed shared
// memory -- one launch, no workspace.  Bound by HBM: the visible cache is read once for
// all query heads of the group.
//
// bf16: warp-level matrix instructions over 16 heads x 16 keys (8 heads for groups of up
// to 8).  Keys and values are fetched one or two steps ahead, 16 bytes a lane, into a place
// of the lane's own in shared memory, and go from there into operand registers as they are:
// a dot product does not care in which order its channels are taken, so a lane's 16 bytes
// of a key serve as two k-steps of it (the query is loaded in the same order), and an
// output tile takes every eighth channel so that a lane's 16 bytes of a value row feed
// eight tiles.  (The fifth-generation tensor core would not be used a tenth: a step of 16
// keys is 64 warp instructions here against 8 KB from memory.)
// 256 sequences of 2052 positions, 16 query heads of 128 over 4: 214 us (5.0 TB/s) call after
// call in a graph, 232 with the caches of other sequences in between; over 16: 775 us, 5.6
// TB/s; one sequence: 9 us in a graph.  Heads of 64: 113 over 4, 405 over 16.  What is left of
// the first is the CTAs' own beginning and end (position, query, first rows; join), about 10
// us a wave: three CTAs of an SM overlap it (with two, and twice the bytes in flight, 231 us).
// fp32: one key row per half or whole warp on the CUDA cores, up to four heads of a group a
// CTA; 64 sequences of 2052 positions, 8 heads of 128 over 8: 174 us (6.2 TB/s), 16 over 4: 185,
// 32 over 4 (whose cache is read twice): 328.
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
__device__ __forceinline__ void copy16(uint32_t smem, const void *p, uint32_t bytes = 16)  // (16, or 0: zeros arrive)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_group_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_groups_wait()  // all but the last N
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Keys and values on their way: AHEAD steps of 16 rows of each a warp, every 16 bytes in
// the place of the lane that asked for them and will use them (so no barrier is needed).
// The warps' results take the same room afterwards.
template <int NW, int GC, int D, int AHEAD>
struct MmaShared {
    static constexpr int STEP = 16 * D * 2;  // bytes of 16 rows
    union {
        uint8_t ring[NW][2 * AHEAD][STEP];
        Partials<NW, GC, D> part;
    };
    Joined<GC, D> joined;
};

// HR x 8 query heads of a CTA: both halves of the matrix instruction's rows, or one (whose
// registers then let a third or fourth CTA onto the SM).  PER_SM CTAs on an SM.
template <int D, int HR, int NW, int AHEAD, int PER_SM>
__global__ void __launch_bounds__(NW * 32, PER_SM) decode_mma_kernel(const SwaDecodeArgs a, int nsplit, int nchunk)
{
    using E = __nv_bfloat16;
    constexpr int kHeads = 8 * HR;
    constexpr int NC = D / 32;  // 16-byte chunks of a row per lane
    using Shared = MmaShared<NW, kHeads, D, AHEAD>;
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
    // rows behind the run stand at its last position again: their scores are masked, and their
    // values are zeros (an infinity that the last position holds would meet their weight of 0)
    auto row = [&](const E *fresh, const E *cache, int t) {
        const int p = vis.position(t < t1 ? t : t1 - 1);
        return p == P ? fresh : cache + vis.slot(p) * cstep;
    };
    const uint8_t *ring = &reinterpret_cast<Shared *>(dyn)->ring[warp][0][0] + lane * 16;
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
    auto fetch_keys = [&](int t, int slot) {
        if (t < t1) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const E *p = row(kn, kc, t + gr + 8 * r) + c * 8;
#pragma unroll
                for (int j = 0; j < NC; ++j) copy16(ring_at + slot * Shared::STEP + (r * NC + j) * 512, p + j * 32);
            }
        }
        copy_group_end();
    };
    auto fetch_values = [&](int t, int slot) {
        if (t < t1) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int tr = t + 2 * c + (r & 1) + (r >> 1) * 8;
                const E *p = row(vn, vc, tr) + gr * 8;
#pragma unroll
                for (int j = 0; j < D / 64; ++j)
                    copy16(ring_at + (AHEAD + slot) * Shared::STEP + (r * (D / 64) + j) * 512, p + j * 64, tr < t1 ? 16 : 0);
            }
        }
        copy_group_end();
    };
    auto at = [&](int slot, int n) { return *reinterpret_cast<const uint4 *>(ring + slot * Shared::STEP + n * 512); };
    float m[HR], l[HR] = {}, o[D / 8][2 * HR] = {};
#pragma unroll
    for (int h = 0; h < HR; ++h) m[h] = -INFINITY;
    const float sc = a.scale * kLog2E;
    int t = t0 + warp * 16;
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) {
        fetch_keys(t + n * NW * 16, n);
        fetch_values(t + n * NW * 16, n);
    }
    for (int slot = 0; t < t1; t += NW * 16, slot = slot + 1 == AHEAD ? 0 : slot + 1) {
        float s[2][2 * HR] = {};
        copy_groups_wait<2 * AHEAD - 1>();
        uint4 kf[2][NC];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int j = 0; j < NC; ++j) kf[r][j] = at(slot, r * NC + j);
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
        fetch_keys(t + AHEAD * NW * 16, slot);  // (behind the products, which have read the slot)
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
        copy_groups_wait<2 * AHEAD - 1>();
        uint4 vf[4][D / 64];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < D / 64; ++j) vf[r][j] = at(AHEAD + slot, r * (D / 64) + j);
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
        fetch_values(t + AHEAD * NW * 16, slot);
    }
    copy_groups_wait<0>();
    __syncthreads();  // the warps' results go over the rings
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

// GC query heads of a group and NW warps per CTA.
//
// CTAs that share a (sequence, heads) row: the number with the least waves x time of a
// CTA, whose own cost (query, join, cluster) counts as much as about 300 positions (256 x 4
// rows of 2052 positions of 128 bf16: 234 us in 1, 217 in 2, 230 in 3, 239 in 4, 260 in 6).
// A wave is as many clusters as the device holds at once, which it is asked for: a cluster
// lies within a group of SMs, and where one CTA fills an SM only 15 clusters of 8 fit the
// 148 SMs (16 rows: 16.8 us in 8, 11.2 in 6).  Odd numbers leave more SMs of a group idle
// and are not tried (64 x 4 rows: 66 us in 3, 60 in 1).
template <auto kern, int GC, int NW, typename Shared>
cudaError_t launch(const SwaDecodeArgs &a, cudaStream_t stream)
{
    static std::atomic<unsigned long long> set{0};
    static std::atomic<int> fit[kMaxSplit];  // clusters of n + 1 that fit (the kernels are sm_100a's: the same on every device)
    cudaError_t e = ensure_smem_limit(kern, sizeof(Shared), set);
    if (e != cudaSuccess) return e;
    const int G = a.Hq / a.Hk, nchunk = (G + GC - 1) / GC;
    const long long rows = (long long)a.B * a.Hk * nchunk, seen = (long long)a.window + a.sinks;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(NW * 32);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int nsplit = 1;
    double least = 0;
    for (int n = 1; n <= kMaxSplit; n += n == 1 ? 1 : 2) {
        int m = fit[n - 1].load(std::memory_order_relaxed);
        if (m == 0) {
            attr[0].val.clusterDim.x = n;
            cfg.gridDim = dim3(n);
            if ((e = cudaOccupancyMaxActiveClusters(&m, kern, &cfg)) != cudaSuccess) return e;
            if (m < 1) m = 1;
            fit[n - 1].store(m, std::memory_order_relaxed);
        }
        const double cost = (double)((rows + m - 1) / m) * ((double)seen / n + 300.0);
        if (n == 1 || cost < least) least = cost, nsplit = n;
    }
    attr[0].val.clusterDim.x = nsplit;
    cfg.gridDim = dim3(nsplit, a.Hk * nchunk, a.B);  // (y is at most the number of query heads)
    cfg.numAttrs = nsplit > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a, nsplit, nchunk);
}

template <int D, int HR, int NW, int AHEAD, int PER_SM>
cudaError_t launch_mma(const SwaDecodeArgs &a, cudaStream_t stream)
{
    return launch<decode_mma_kernel<D, HR, NW, AHEAD, PER_SM>, 8 * HR, NW, MmaShared<NW, 8 * HR, D, AHEAD>>(a, stream);
}

template <int D>
cudaError_t by_group_f32(const SwaDecodeArgs &a, cudaStream_t stream)
{
    const int G = a.Hq / a.Hk;
    if (G == 1) return launch<decode_kernel<float, D, 1>, 1, 4, DecodeShared<4, 1, D>>(a, stream);
    if (G == 2) return launch<decode_kernel<float, D, 2>, 2, 4, DecodeShared<4, 2, D>>(a, stream);
    return launch<decode_kernel<float, D, 4>, 4, 4, DecodeShared<4, 4, D>>(a, stream);
}

}  // namespace

cudaError_t launch_swa_decode(const SwaDecodeArgs &a, bool bf16, int num_sms, cudaStream_t stream)
{
    if (bf16) {
        // few rows: eight warps a CTA, so that a warp's walk is short (one sequence, 16 heads of
        // 128, 2052 slots: 11.0 us, and 13.8 with four).  Else as many CTAs on an SM as the
        // registers allow without spilling (four of 128 threads at d = 128 spill: 292 us
        // against 216 with three).
        const bool small_group = a.Hq / a.Hk <= 8;
        if (small_group && (long long)a.B * a.Hk * kMaxSplit <= num_sms)
            return a.d == 128 ? launch_mma<128, 1, 8, 2, 1>(a, stream) : launch_mma<64, 1, 8, 2, 1>(a, stream);
        if (small_group)
            return a.d == 128 ? launch_mma<128, 1, 4, 1, 3>(a, stream) : launch_mma<64, 1, 4, 2, 4>(a, stream);
        return a.d == 128 ? launch_mma<128, 2, 4, 2, 2>(a, stream) : launch_mma<64, 2, 4, 2, 4>(a, stream);
    }
    return a.d == 128 ? by_group_f32<128>(a, stream) : by_group_f32<64>(a, stream);
}

}  // namespace gdn2
