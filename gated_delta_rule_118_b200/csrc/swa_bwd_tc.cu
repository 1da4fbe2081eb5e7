// swa_bwd_tc.cu -- windowed attention backward for bf16 on the tensor cores.
//
// Two kernels, so that every sum has one owner and a fixed order (no atomics): dk and dv
// by key tiles, dq by query tiles.  Scores and dO v^T are formed in both (7 products of
// 128 x 128 x d a tile pair instead of 5).  In both kernels the matrix that a product
// reads as its left operand (P^T, dS^T, or dS) is written as bf16 straight into tensor
// memory over the fp32 values it came from, so nothing but the inputs passes through
// shared memory:
//   dk, dv:  S^T = K Q^T,  dP^T = V dO^T     one key row per thread pair (64 queries each)
//            P^T = exp(scale S^T - lse),  dS^T = P^T (dP^T - delta)
//            dV += P^T dO,  dK += dS^T Q
//   dq:      S = Q K^T,  dP = dO V^T,  dS = P (dP - delta),  dQ += dS K
// P is rounded to bf16 (2^-8 relative at most, as the operand of a bf16 product).  dS goes
// in as the sum of two bf16 matrices, 16 bits together: rounded once, its error is as large
// as that of the rounding on the way out (relative error of dq 2.5e-3 with one, 1.8e-3 with
// two, 1.7e-3 being the outputs' own; two more products of nine cost 13 % of the time).
// Scores, probabilities' exponents, sums and gradients are fp32 up to the one rounding on
// the way out.
//
// Bound by the tensor pipe and the hand-overs around it: 4 x 4096, 16 query heads of 128
// over 4, window 2048, 4 sinks: 890 to 980 us from one device to another, dk and dv a little
// more of it than dq (tensor pipe active 60 % and 52 % of the time); 1 x 16384 x 16 heads 1160
// to 1320 us.  One thread issues the products of dk and dv (with a warp for those of P and one
// for those of dS 1224 us against 1197: each delays the other's), and one each those of scores
// and of dq (1197 against 1222).
//
// Keys that every later row sees (sinks) have as many query tiles as the sequence;
// where that would leave a few CTAs with most of the work, their query range is split
// into segments whose fp32 partial sums a small kernel adds in order.
#include <cuda.h>

#include "launch.h"
#include "sm100.cuh"
#include "swa_common.cuh"
#include "tc_common.cuh"

namespace gdn2 {
namespace {

using namespace swa;
using namespace sm100;

constexpr int kThreads = 384;  // two warpgroups that compute, then the issuing warps
constexpr int kTma = 8, kMma = 9, kRows = 10;
// 384 threads launch with 168 registers each: 2 x 128 x 208 + 128 x 88 = 384 x 168
constexpr int kRegsCompute = 208, kRegsIssue = 88;

template <int D>
struct Tiles {
    static constexpr int TILE = 128 * D * 2;  // bytes of a 128-row tile, boxes of 64 channels
    static constexpr uint32_t STEP = TILE >> 4;
};

template <int D>
__device__ __forceinline__ void load_tile(uint8_t *dst, const CUtensorMap *m, uint64_t *bar, int h, int row, int b)
{
    for (int x = 0; x < D / 64; ++x) tma_load_4d(dst + x * 16384, m, bar, x * 64, h, row, b);
}

// D[128 x 128] = A B^T over d: both tiles in shared memory, rows of d.
template <int D>
__device__ __forceinline__ void issue_rows(uint32_t tm, uint64_t da, uint64_t db)
{
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t o = (ks >> 2) * 1024 + (ks & 3) * 2;
        umma_bf16(tm, da + o, db + o, idesc_bf16(128, 128, 0, 0), ks > 0);
    }
}
// D[128 x d] += A B: A bf16 in tensor memory (128 columns, 64 of them from tm_a, 64 from
// tm_a + 64), B a tile of 128 rows of d.  PAIR: A is a sum of two such matrices, the
// second 32 columns behind the first.
template <int D, bool PAIR>
__device__ __forceinline__ void issue_cols(uint32_t tm, uint32_t tm_a, uint64_t db, uint32_t acc)
{
#pragma unroll
    for (int x = 0; x <= (int)PAIR; ++x)
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
            umma_bf16_ts(tm, tm_a + x * 32 + (ks >> 2) * 64 + (ks & 3) * 8, db + ks * 128, idesc_bf16(128, D, 0, 1), acc | (x + ks > 0));
}

// 64 values packed to bf16 over the columns they came from.
__device__ __forceinline__ void put_bf16(uint32_t tm, const float (&f)[64])
{
    uint32_t u[32];
#pragma unroll
    for (int x = 0; x < 64; x += 2) {
        const __nv_bfloat162 e = __floats2bfloat162_rn(f[x], f[x + 1]);
        u[x / 2] = *reinterpret_cast<const uint32_t *>(&e);
    }
    tmem_st32(tm, u);
    tmem_st_wait();
    tc_fence_before();
}

// The same as a sum of two: the upper half of each value's bits (cut off, which takes no
// conversion), and 32 columns behind what that leaves, rounded.  Together they carry 16
// bits.
__device__ __forceinline__ void put_bf16_pair(uint32_t tm, const float (&f)[64])
{
#pragma unroll
    for (int y = 0; y < 64; y += 32) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int x = 0; x < 32; x += 2) {
            const uint32_t a = __float_as_uint(f[y + x]), b = __float_as_uint(f[y + x + 1]);
            hi[x / 2] = __byte_perm(a, b, 0x7632);
            const __nv_bfloat162 r = __floats2bfloat162_rn(f[y + x] - __uint_as_float(a & 0xffff0000u),
                                                           f[y + x + 1] - __uint_as_float(b & 0xffff0000u));
            lo[x / 2] = *reinterpret_cast<const uint32_t *>(&r);
        }
        tmem_st16(tm + y / 2, hi);
        tmem_st16(tm + 32 + y / 2, lo);
    }
    tmem_st_wait();
    tc_fence_before();
}

// Half a row (D / 2 columns from tm) scaled and written, or zeros where not `live`; true
// if something is not finite.  `have` (the same in the whole warp): there are values in tm.
template <int D, typename E>
__device__ __forceinline__ bool put_row(uint32_t tm, float f, E *dst, bool inside, bool live, bool have)
{
    bool bad = false;
#pragma unroll
    for (int x = 0; x < D / 2; x += 32) {
        float o[32];
        if (have) {
            tmem_ld32(tm + x, o);
            tmem_ld_wait(o);
        }
#pragma unroll
        for (int y = 0; y < 32; ++y) {
            o[y] = have && live ? o[y] * f : 0.f;
            bad |= !isfinite(o[y]);
        }
        if (inside)
#pragma unroll
            for (int y = 0; y < 32; y += 4) store4(dst + x + y, make_float4(o[y], o[y + 1], o[y + 2], o[y + 3]));
    }
    return bad && inside;
}

// ---------------------------------------------------------------- dk, dv
// The work of one CTA along grid z (slowest, so that the long ranges of all heads start
// first): a key tile and its range of query tiles.
struct KvPlan {
    int nseg;      // segments of a sink tile's queries; 0: no splitting
    int seg;       // query tiles of a segment
    int nsink;     // key tiles with sinks
    int ntiles;    // key tiles
    float *part;   // [B][Hk][nsink][nseg][2][128][d] partial sums
};

struct KvRange {
    int j0, q0, q1, slot;  // first key, query tiles [q0, q1), partial slot (-1: final)
    __device__ __forceinline__ KvRange(const SwaArgs &a, const KvPlan &p, int x, int n)
    {
        const int off = a.Tk - a.T, split = p.nseg ? p.nsink * p.nseg : 0;
        slot = x < split ? x : -1;
        const int tile = x < split ? x / p.nseg : x - split + (p.nseg ? p.nsink : 0);
        j0 = tile * 128;
        q0 = (j0 > off ? j0 - off : 0) >> 7;
        const long long far = (long long)min(j0 + 128, a.Tk) - 1 + a.window - off;  // first row behind every window
        const int hi = (j0 < a.sinks || far > n) ? n : far < 0 ? 0 : (int)far;
        q1 = (hi + 127) >> 7;
        if (slot >= 0) {
            q0 += x % p.nseg * p.seg;
            q1 = min(q1, q0 + p.seg);
        }
    }
};

enum { KV_FULL, QG_FULL, QG_EMPTY = QG_FULL + 2, EXT_FULL = QG_EMPTY + 2, S_FULL = EXT_FULL + 2, DP_FULL, P_FULL, DS_FULL,
       DONE, NBAR };

template <int D>
struct KvLayout {
    static constexpr int TILE = Tiles<D>::TILE;
    static constexpr int K = 0, V = TILE, Q = 2 * TILE, G = 4 * TILE;
    // the sixteen more steps of the inner products that subtract lse and delta: 16-byte rows
    // of eight steps, [stage][lse, delta][128 rows]; the key tile's; eight steps of zeros
    static constexpr int EXT = 6 * TILE, MINUS = EXT + 4 * 2048, ZERO = MINUS + 2048;
    static constexpr int BADS = ZERO + 2048;      // [half][128]
    static constexpr int BAR = BADS + 1024;
    static constexpr int SLOT = BAR + 8 * NBAR + 8;
    __host__ __device__ static constexpr int ext(int stage, int which) { return EXT + (stage * 2 + which) * 2048; }
    static constexpr int BYTES = SLOT + 16 + 1024;
    static constexpr uint32_t TM_S = 0, TM_DP = 128, TM_DV = 256, TM_DK = 256 + D;
};

template <int D, bool LENS>
__global__ void __launch_bounds__(kThreads, 1)
dkdv_tc_kernel(const __grid_constant__ SwaArgs a, const KvPlan plan, const __grid_constant__ CUtensorMap mq,
               const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
               const __grid_constant__ CUtensorMap mg)
{
    using L = KvLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hk = blockIdx.x, b = blockIdx.y;
    const int n = seq_len(a, b), off = a.Tk - a.T, G = a.Hq / a.Hk;
    const KvRange rg(a, plan, blockIdx.z, n);
    const int nq = max(rg.q1 - rg.q0, 0), N = G * nq;
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::BAR);
    uint32_t *slot = reinterpret_cast<uint32_t *>(sm + L::SLOT);
    if (tid == 0) {
        for (int i = 0; i < NBAR; ++i) mbar_init(bar + i, i == P_FULL || i == DS_FULL ? 8 : 1);
        fence_mbar_init();
    }
    if (tid < 128) {  // the key tile's further steps: -1 against the three parts of lse or delta
        const uint32_t m1 = 0xbf80bf80u;
        *reinterpret_cast<uint4 *>(sm + L::ZERO + tid * 16) = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4 *>(sm + L::MINUS + tid * 16) = make_uint4(m1, m1 & 0xffffu, 0, 0);
        fence_proxy_async_smem();
    }
    if (warp == kMma) {
        tmem_alloc(slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot;
    const uint32_t sbase = smem_u32(sm);
    // the walk over (head, query tile)
    struct Walk {
        int h, q, q0, q1;
        __device__ __forceinline__ void next() { if (++q == q1) q = q0, ++h; }
    };
    const Walk start{hk * G, rg.q0, rg.q0, rg.q1};

    if (warp >= 8) {
        setmaxnreg_dec<kRegsIssue>();
        if (warp == kTma && N > 0) {
            if (elect_one()) {
                mbar_arrive_expect_tx(bar + KV_FULL, 2 * L::TILE);
                load_tile<D>(sm + L::K, &mk, bar + KV_FULL, hk, rg.j0, b);
                load_tile<D>(sm + L::V, &mv, bar + KV_FULL, hk, rg.j0, b);
            }
            __syncwarp();
            int i = 0;
            Walk w = start;
            for (; i < N; ++i, w.next()) {
                const int s = i & 1;
                if (!__all_sync(~0u, mbar_wait(bar + QG_EMPTY + s, ((i >> 1) & 1) ^ 1, a.err))) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(bar + QG_FULL + s, 2 * L::TILE);
                    load_tile<D>(sm + L::Q + s * L::TILE, &mq, bar + QG_FULL + s, w.h, w.q * 128, b);
                    load_tile<D>(sm + L::G + s * L::TILE, &mg, bar + QG_FULL + s, w.h, w.q * 128, b);
                }
                __syncwarp();
            }
            // every copy has landed before the CTA ends, also when another role gave up
            mbar_wait(bar + KV_FULL, 0, a.err);
            for (int c = max(i - 2, 0); c < i; ++c) mbar_wait(bar + QG_FULL + (c & 1), (c >> 1) & 1, a.err);
        } else if (warp == kRows) {
            // lse / scale and delta of the tile's rows, each as three bf16 parts (their sum is
            // within 2^-24 of it), subtracted by the products themselves.  Rows without a token
            // or without a finite score get 2^100, so that their probabilities come out 0.
            auto split = [](float x) {
                const float hi = __bfloat162float(__float2bfloat16_rn(x)), mid = __bfloat162float(__float2bfloat16_rn(x - hi));
                const __nv_bfloat162 u = __floats2bfloat162_rn(hi, mid);
                const uint32_t lo = __bfloat16_as_ushort(__float2bfloat16_rn((x - hi) - mid));
                return make_uint4(*reinterpret_cast<const uint32_t *>(&u), lo, 0, 0);
            };
            const float inv = 1.f / a.scale;
            Walk w = start;
            for (int i = 0; i < N; ++i, w.next()) {
                const int s = i & 1;
                const long long at = ((long long)b * a.Hq + w.h) * a.T;
                float l[4], d[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int row = w.q * 128 + x * 32 + lane;
                    l[x] = row < n ? a.lse[at + row] : -INFINITY;
                    d[x] = row < n ? a.delta[at + row] : 0.f;
                }
                if (!__all_sync(~0u, mbar_wait(bar + QG_EMPTY + s, ((i >> 1) & 1) ^ 1, a.err))) break;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    *reinterpret_cast<uint4 *>(sm + L::ext(s, 0) + (x * 32 + lane) * 16) =
                        l[x] == -INFINITY ? make_uint4(0x7180u, 0, 0, 0) : split(l[x] * inv);
                    *reinterpret_cast<uint4 *>(sm + L::ext(s, 1) + (x * 32 + lane) * 16) = split(d[x]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                const int rows = n - w.q * 128;  // behind them is padding
                if (LENS && n < a.T && rows < 128) {
                    if (!__all_sync(~0u, mbar_wait(bar + QG_FULL + s, (i >> 1) & 1, a.err))) break;
                    zero_rows<D>(sm + L::Q + s * L::TILE, rows);
                    zero_rows<D>(sm + L::G + s * L::TILE, rows);
                }
                if (lane == 0) mbar_arrive(bar + EXT_FULL + s);
            }
        } else if (warp == kMma && N > 0) {
            const uint64_t dk = smem_desc(sbase + L::K, 16, 1024, kSw128), dv = smem_desc(sbase + L::V, 16, 1024, kSw128);
            const uint64_t dq = smem_desc(sbase + L::Q, 16, 1024, kSw128), dg = smem_desc(sbase + L::G, 16, 1024, kSw128);
            const uint64_t qt = smem_desc(sbase + L::Q, 16384, 1024, kSw128), gt = smem_desc(sbase + L::G, 16384, 1024, kSw128);
            constexpr uint32_t STEP = Tiles<D>::STEP;
            const uint64_t minus = smem_desc(sbase + L::MINUS, (uint32_t)(L::ZERO - L::MINUS), 128, kSwNone);
            // S^T less lse / scale, and dP^T less delta, of stage s
            auto scores = [&](uint32_t s) {
                issue_rows<D>(tmem + L::TM_S, dk, dq + s * STEP);
                umma_bf16(tmem + L::TM_S, minus, smem_desc(sbase + L::ext(s, 0), L::ZERO - L::ext(s, 0), 128, kSwNone),
                          idesc_bf16(128, 128, 0, 0), 1);
                umma_commit(bar + S_FULL);
            };
            auto dots = [&](uint32_t s) {
                issue_rows<D>(tmem + L::TM_DP, dv, dg + s * STEP);
                umma_bf16(tmem + L::TM_DP, minus, smem_desc(sbase + L::ext(s, 1), L::ZERO - L::ext(s, 1), 128, kSwNone),
                          idesc_bf16(128, 128, 0, 0), 1);
                umma_commit(bar + DP_FULL);
            };
            bool ok = mbar_wait(bar + KV_FULL, 0, a.err) && mbar_wait(bar + QG_FULL, 0, a.err) && mbar_wait(bar + EXT_FULL, 0, a.err);
            ok = __all_sync(~0u, ok);
            if (ok) {
                tc_fence_after();
                if (elect_one()) {
                    scores(0);
                    dots(0);
                }
                __syncwarp();
            }
            for (int i = 0; ok && i < N; ++i) {
                const uint32_t s = i & 1, sn = s ^ 1;
                const bool next = i + 1 < N;
                if (next)
                    ok = mbar_wait(bar + QG_FULL + sn, ((i + 1) >> 1) & 1, a.err) && mbar_wait(bar + EXT_FULL + sn, ((i + 1) >> 1) & 1, a.err);
                ok = __all_sync(~0u, ok && mbar_wait(bar + P_FULL, s, a.err));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    issue_cols<D, false>(tmem + L::TM_DV, tmem + L::TM_S, gt + s * STEP, i > 0);
                    if (next) scores(sn);  // over P^T, which the product just issued reads: products run in order
                }
                __syncwarp();
                ok = __all_sync(~0u, mbar_wait(bar + DS_FULL, s, a.err));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    issue_cols<D, true>(tmem + L::TM_DK, tmem + L::TM_DP, qt + s * STEP, i > 0);
                    umma_commit(bar + QG_EMPTY + s);
                    if (next) dots(sn);
                }
                __syncwarp();
            }
            if (elect_one()) umma_commit(bar + DONE);
            __syncwarp();
            mbar_wait(bar + DONE, 0, a.err);  // no product is in flight when the tensor memory is freed
        }
    } else {
        setmaxnreg_inc<kRegsCompute>();
        const int hf = warp >> 2, r = tid & 127, j = rg.j0 + r;
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t ts = lane_base + L::TM_S + hf * 64, tp = lane_base + L::TM_DP + hf * 64;
        const float sc = a.scale * kLog2E;
        bool ok = true;
        // query tiles whose rows all hold a token and see all of these keys: first rows [lo, hi]
        const int full_lo = rg.j0 + 127 - off;
        const int full_hi = rg.j0 + 128 <= a.sinks ? n - 128 : min(n - 128, a.window - 128 + rg.j0 - off);
        Walk w = start;
        for (int i = 0; i < N; ++i, w.next()) {
            const int s = i & 1, i0 = w.q * 128;
            ok = __all_sync(~0u, mbar_wait(bar + S_FULL, s, a.err));
            if (!ok) break;
            tc_fence_after();
            float p[64];
            tmem_ld32(ts, *reinterpret_cast<float(*)[32]>(p));
            tmem_ld32(ts + 32, *reinterpret_cast<float(*)[32]>(p + 32));
            tmem_ld_wait(p);
            const bool full = i0 >= full_lo && i0 <= full_hi;
            if (__builtin_expect(!full, 0)) {
                // (rows behind the length have p = 0 by their lse, but what stands in their q
                // and dO must not reach the exponential or the product with it)
                const int c0 = i0 + hf * 64, lo = j - off - c0;
                const long long far = (long long)lo + a.window;
                const int hi = j < a.sinks || far > n - c0 ? n - c0 : (int)far;
#pragma unroll
                for (int x = 0; x < 64; ++x) p[x] = x >= lo && x < hi ? p[x] : -INFINITY;
            }
#pragma unroll
            for (int x = 0; x < 64; ++x) p[x] = ex2_approx(p[x] * sc);
            put_bf16(ts, p);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + P_FULL);
            ok = __all_sync(~0u, mbar_wait(bar + DP_FULL, s, a.err));
            if (!ok) break;
            tc_fence_after();
            float g[64];
            tmem_ld32(tp, *reinterpret_cast<float(*)[32]>(g));
            tmem_ld32(tp + 32, *reinterpret_cast<float(*)[32]>(g + 32));
            tmem_ld_wait(g);
            if (__builtin_expect(!full, 0)) {
#pragma unroll
                for (int x = 0; x < 64; ++x) g[x] = p[x] == 0.f ? 0.f : g[x];
            }
#pragma unroll
            for (int x = 0; x < 64; ++x) g[x] *= p[x];
            put_bf16_pair(tp, g);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + DS_FULL);
        }
        if (ok && N > 0) ok = mbar_wait(bar + DONE, 0, a.err);
        ok = named_bar_and(1, 256, ok);
        tc_fence_after();
        if (ok) {
            const uint32_t tv = lane_base + L::TM_DV + hf * (D / 2), tk = lane_base + L::TM_DK + hf * (D / 2);
            const bool have = N > 0, inside = j < a.Tk;
            if (rg.slot >= 0) {  // partial sums of a segment
                float *part = plan.part + ((((long long)b * a.Hk + hk) * plan.nsink * plan.nseg + rg.slot) * 256 + r) * D + hf * (D / 2);
                put_row<D>(tk, a.scale, part, true, true, have);
                put_row<D>(tv, 1.f, part + 128 * D, true, true, have);
            } else {
                const long long at = (((long long)b * a.Tk + j) * a.Hk + hk) * D + hf * (D / 2);
                bool bad = put_row<D>(tk, a.scale, static_cast<bf16 *>(a.dk) + at, inside, true, have);
                bad |= put_row<D>(tv, 1.f, static_cast<bf16 *>(a.dv) + at, inside, true, have);
                uint32_t *bads = reinterpret_cast<uint32_t *>(sm + L::BADS);
                bads[hf * 128 + r] = bad;
                named_bar(1, 256);
                unsigned todo = __ballot_sync(~0u, bads[r] | bads[128 + r]) & (hf ? 0xffff0000u : 0xffffu);
                while (todo) {
                    const int r0 = __ffs(todo) - 1;
                    todo &= todo - 1;
                    row_dkdv<bf16, D>(a, b, hk, j - lane + r0);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// dk and dv of the sink tiles: the segments' partial sums added in order, one warp a key.
template <int D>
__global__ void __launch_bounds__(256) sink_sum_kernel(const __grid_constant__ SwaArgs a, const KvPlan plan)
{
    const int j = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31, hk = blockIdx.y, b = blockIdx.z;
    if (j >= plan.nsink * 128 || j >= a.Tk) return;
    const float *part = plan.part + ((((long long)b * a.Hk + hk) * plan.nsink + (j >> 7)) * plan.nseg * 256 + (j & 127)) * D;
    bool bad = false;
    float v[2][D / 32] = {};
    for (int s = 0; s < plan.nseg; ++s)
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int u = 0; u < D / 32; ++u) v[w][u] += part[((long long)s * 256 + w * 128) * D + lane + 32 * u];
    const long long at = (((long long)b * a.Tk + j) * a.Hk + hk) * D;
#pragma unroll
    for (int u = 0; u < D / 32; ++u) {
        bad |= !isfinite(v[0][u]) || !isfinite(v[1][u]);
        static_cast<bf16 *>(a.dk)[at + lane + 32 * u] = __float2bfloat16_rn(v[0][u]);
        static_cast<bf16 *>(a.dv)[at + lane + 32 * u] = __float2bfloat16_rn(v[1][u]);
    }
    if (__any_sync(~0u, bad)) row_dkdv<bf16, D>(a, b, hk, j);
}

// ---------------------------------------------------------------- dq
enum { QD_FULL, K_FULL, K_EMPTY = K_FULL + 3, V_FULL = K_EMPTY + 3, V_EMPTY, SQ_FULL, SQ_FREE,
       DPQ_FULL, DSQ_FULL = DPQ_FULL + 2, DQ_DONE = DSQ_FULL + 2, SCORES_DONE = DQ_DONE + 2, DONE_Q, NBAR_Q };

template <int D>
struct QLayout {
    static constexpr int TILE = Tiles<D>::TILE;
    // three stages of K, which dQ reads last, and one of V, which only dP reads
    static constexpr int Q = 0, G = TILE, K = 2 * TILE, V = 5 * TILE;
    static constexpr int BAD = 6 * TILE;           // [half][128]
    static constexpr int BAR = BAD + 1024;
    static constexpr int SLOT = BAR + 8 * NBAR_Q + 8;
    static constexpr int BYTES = SLOT + 16 + 1024;
    static constexpr uint32_t TM_S = 0, TM_DP = 128, TM_DQ = 384;  // two buffers of dP
};

template <int D, bool LENS>
__global__ void __launch_bounds__(kThreads, 1)
dq_tc_kernel(const __grid_constant__ SwaArgs a, const __grid_constant__ CUtensorMap mq,
             const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
             const __grid_constant__ CUtensorMap mg)
{
    using L = QLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int i0 = (gridDim.z - 1 - blockIdx.z) * 128, h = blockIdx.x, b = blockIdx.y;  // longest rows first
    const int n = seq_len(a, b), off = a.Tk - a.T, hk = h / (a.Hq / a.Hk);
    if (i0 >= n) {  // padding only
        const int rows = min(128, a.T - i0);
        bf16 *out = static_cast<bf16 *>(a.dq) + (((long long)b * a.T + i0) * a.Hq + h) * D;
        for (int c = tid; c < rows * (D / 8); c += kThreads)
            *reinterpret_cast<uint4 *>(out + (long long)(c / (D / 8)) * a.Hq * D + c % (D / 8) * 8) = make_uint4(0, 0, 0, 0);
        return;
    }
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::BAR);
    uint32_t *slot = reinterpret_cast<uint32_t *>(sm + L::SLOT);
    if (tid == 0) {
        for (int i = 0; i < NBAR_Q; ++i) mbar_init(bar + i, i == SQ_FREE || i == DSQ_FULL || i == DSQ_FULL + 1 ? 8 : 1);
        fence_mbar_init();
    }
    if (warp == kMma) {
        tmem_alloc(slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot;
    const uint32_t sbase = smem_u32(sm);
    const KeyTiles kt(off + i0, off + min(i0 + 128, n) - 1, a.window, a.sinks, 128);
    const int N = kt.count();

    if (warp >= 8) {
        setmaxnreg_dec<kRegsIssue>();
        if (warp == kTma) {
            if (elect_one()) {
                mbar_arrive_expect_tx(bar + QD_FULL, 2 * L::TILE);
                load_tile<D>(sm + L::Q, &mq, bar + QD_FULL, h, i0, b);
                load_tile<D>(sm + L::G, &mg, bar + QD_FULL, h, i0, b);
            }
            __syncwarp();
            int nk = 0, nv = 0, ks = 0;
            uint32_t kph = 1;
            for (int c = 0; c < N; ++c) {
                if (!__all_sync(~0u, mbar_wait(bar + K_EMPTY + ks, kph, a.err))) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(bar + K_FULL + ks, L::TILE);
                    load_tile<D>(sm + L::K + ks * L::TILE, &mk, bar + K_FULL + ks, hk, kt.tile(c) * 128, b);
                }
                __syncwarp();
                nk = c + 1;
                if (!__all_sync(~0u, mbar_wait(bar + V_EMPTY, (c & 1) ^ 1, a.err))) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(bar + V_FULL, L::TILE);
                    load_tile<D>(sm + L::V, &mv, bar + V_FULL, hk, kt.tile(c) * 128, b);
                }
                __syncwarp();
                nv = c + 1;
                if (++ks == 3) ks = 0, kph ^= 1;
            }
            // every copy has landed before the CTA ends, also when another role gave up
            mbar_wait(bar + QD_FULL, 0, a.err);
            for (int c = max(nk - 3, 0); c < nk; ++c) mbar_wait(bar + K_FULL + c % 3, (c / 3) & 1, a.err);
            if (nv > 0) mbar_wait(bar + V_FULL, (nv - 1) & 1, a.err);
        } else if (warp == kMma) {
            const uint64_t dq = smem_desc(sbase + L::Q, 16, 1024, kSw128), dg = smem_desc(sbase + L::G, 16, 1024, kSw128);
            const uint64_t dk = smem_desc(sbase + L::K, 16, 1024, kSw128), dv = smem_desc(sbase + L::V, 16, 1024, kSw128);
            constexpr uint32_t STEP = Tiles<D>::STEP;
            bool ok = __all_sync(~0u, mbar_wait(bar + QD_FULL, 0, a.err));
            uint32_t ks = 0, kph = 0;  // K stage
            for (int c = 0; ok && c < N; ++c) {
                // S and dP of tile c; S goes over the S that has been read, dP over dS of the tile
                // before last, which its product has read
                const uint32_t s = c & 1;
                ok = mbar_wait(bar + K_FULL + ks, kph, a.err);
                if (c > 0) ok = ok && mbar_wait(bar + SQ_FREE, s ^ 1, a.err);
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    issue_rows<D>(tmem + L::TM_S, dq, dk + ks * STEP);
                    umma_commit(bar + SQ_FULL);
                }
                __syncwarp();
                ok = mbar_wait(bar + V_FULL, s, a.err);
                if (c > 1) ok = ok && mbar_wait(bar + DQ_DONE + s, ((c >> 1) & 1) ^ 1, a.err);
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    issue_rows<D>(tmem + L::TM_DP + s * 128, dg, dv);
                    umma_commit(bar + DPQ_FULL + s);
                    umma_commit(bar + V_EMPTY);
                }
                __syncwarp();
                if (++ks == 3) ks = 0, kph ^= 1;
            }
            if (elect_one()) umma_commit(bar + SCORES_DONE);
            __syncwarp();
            mbar_wait(bar + SCORES_DONE, 0, a.err);  // no product is in flight when the tensor memory is freed
        } else if (warp == kRows) {
            // the products of dQ from a warp of their own: issuing takes about as long as their
            // work, and the next scores would wait for it
            const uint64_t dk = smem_desc(sbase + L::K, 16384, 1024, kSw128);
            bool ok = true;
            uint32_t ks = 0, kph = 0;
            for (int c = 0; c < N; ++c) {
                const uint32_t s = c & 1;
                ok = mbar_wait(bar + K_FULL + ks, kph, a.err) && mbar_wait(bar + DSQ_FULL + s, (c >> 1) & 1, a.err);
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                tc_fence_after();
                // zeros for the padding (the scores, which read this tile too, have been taken)
                if (LENS && c == N - 1 && n < a.T) zero_rows<D>(sm + L::K + ks * L::TILE, min(off + n - kt.tile(c) * 128, 128));
                if (elect_one()) {
                    issue_cols<D, true>(tmem + L::TM_DQ, tmem + L::TM_DP + s * 128, dk + ks * Tiles<D>::STEP, c > 0);
                    umma_commit(bar + DQ_DONE + s);
                    umma_commit(bar + K_EMPTY + ks);
                }
                __syncwarp();
                if (++ks == 3) ks = 0, kph ^= 1;
            }
            if (elect_one()) umma_commit(bar + DONE_Q);
            __syncwarp();
            mbar_wait(bar + DONE_Q, 0, a.err);
        }
    } else {
        setmaxnreg_inc<kRegsCompute>();
        const int hf = warp >> 2, r = tid & 127, row = i0 + r, p_ = off + row;
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const float sc = a.scale * kLog2E;
        const long long lrow = ((long long)b * a.Hq + h) * a.T + row;
        const bool live = row < n;
        const float lse = live ? a.lse[lrow] : -INFINITY, delta = live ? a.delta[lrow] : 0.f;
        const float lse2 = lse == -INFINITY ? INFINITY : lse * kLog2E;
        bool ok = true;
        for (int c = 0; c < N; ++c) {
            const int s = c & 1, j0 = kt.tile(c) * 128;
            const uint32_t tp = lane_base + L::TM_DP + s * 128 + hf * 64;
            ok = __all_sync(~0u, mbar_wait(bar + SQ_FULL, s, a.err));
            if (!ok) break;
            tc_fence_after();
            float p[64];
            tmem_ld32(lane_base + L::TM_S + hf * 64, *reinterpret_cast<float(*)[32]>(p));
            tmem_ld32(lane_base + L::TM_S + hf * 64 + 32, *reinterpret_cast<float(*)[32]>(p + 32));
            tmem_ld_wait(p);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + SQ_FREE);
            const bool full = tile_full(off + i0, off + i0 + 127, j0, j0 + 128, a.window, a.sinks);
            if (__builtin_expect(!full, 0)) {
                const int c0 = j0 + hf * 64, hi = p_ - c0, lo = p_ - a.window + 1 - c0, sk = a.sinks - c0;
#pragma unroll
                for (int x = 0; x < 64; ++x) p[x] = x <= hi && (x >= lo || x < sk) ? p[x] : -INFINITY;
            }
#pragma unroll
            for (int x = 0; x < 64; ++x) p[x] = ex2_approx(fmaf(p[x], sc, -lse2));
            ok = __all_sync(~0u, mbar_wait(bar + DPQ_FULL + s, (c >> 1) & 1, a.err));
            if (!ok) break;
            tc_fence_after();
            float g[64];
            tmem_ld32(tp, *reinterpret_cast<float(*)[32]>(g));
            tmem_ld32(tp + 32, *reinterpret_cast<float(*)[32]>(g + 32));
            tmem_ld_wait(g);
#pragma unroll
            for (int x = 0; x < 64; ++x) g[x] = p[x] * (g[x] - delta);
            if (__builtin_expect(!full, 0)) {
#pragma unroll
                for (int x = 0; x < 64; ++x) g[x] = p[x] == 0.f ? 0.f : g[x];
            }
            put_bf16_pair(tp, g);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + DSQ_FULL + s);
        }
        if (ok) ok = mbar_wait(bar + DONE_Q, 0, a.err);
        ok = named_bar_and(1, 256, ok);
        tc_fence_after();
        if (ok) {
            const long long at = (((long long)b * a.T + row) * a.Hq + h) * D + hf * (D / 2);
            const bool bad = put_row<D>(lane_base + L::TM_DQ + hf * (D / 2), a.scale, static_cast<bf16 *>(a.dq) + at,
                                        row < a.T, live, true);
            uint32_t *bads = reinterpret_cast<uint32_t *>(sm + L::BAD);
            bads[hf * 128 + r] = bad;
            named_bar(1, 256);
            unsigned todo = __ballot_sync(~0u, bads[r] | bads[128 + r]) & (hf ? 0xffff0000u : 0xffffu);
            while (todo) {
                const int r0 = __ffs(todo) - 1;
                todo &= todo - 1;
                row_dq<bf16, D>(a, b, h, row - lane + r0);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// A sink tile's queries are split where the sink tiles alone are fewer CTAs than the
// device has SMs twice over (with more of them they balance by themselves) and a
// sequence has more query tiles than one segment.
KvPlan plan_kv(const SwaArgs &a, int num_sms)
{
    KvPlan p{};
    const int nqt = (a.T + 127) / 128;
    p.ntiles = (a.Tk + 127) / 128;
    p.nsink = (a.sinks + 127) / 128;
    p.seg = nqt / 16 > 16 ? (nqt + 15) / 16 : 16;
    p.nseg = (nqt + p.seg - 1) / p.seg;
    if (p.nseg < 2 || (long long)a.B * a.Hk * p.nsink > 2LL * num_sms) p.nseg = 0;
    return p;
}

// LENS: sequences have lengths, so tiles may hold padding.  (Without them the kernels leave the
// code for it out: 1 x 4096, 16 heads of 128: 252 us, and 257 with it; of 64: 211 and 221.)
template <int D, bool LENS>
cudaError_t impl(const SwaArgs &a, float *part, int num_sms, cudaStream_t stream)
{
    KvPlan plan = plan_kv(a, num_sms);
    plan.part = part;
    static std::atomic<unsigned long long> kv_set{0}, q_set{0};
    cudaError_t e = ensure_smem_limit(dkdv_tc_kernel<D, LENS>, KvLayout<D>::BYTES, kv_set);
    if (e == cudaSuccess) e = ensure_smem_limit(dq_tc_kernel<D, LENS>, QLayout<D>::BYTES, q_set);
    if (e != cudaSuccess) return e;
    const long long gs[3] = {(long long)a.T * a.Hq * D, (long long)a.Hq * D, D};
    CUtensorMap mq, mk, mv, mg;
    if (!make_rows_map(&mq, a.q, D, a.Hq, a.T, a.B, a.qs, 128) || !make_rows_map(&mk, a.k, D, a.Hk, a.Tk, a.B, a.ks, 128) ||
        !make_rows_map(&mv, a.v, D, a.Hk, a.Tk, a.B, a.vs, 128) || !make_rows_map(&mg, a.dO, D, a.Hq, a.T, a.B, gs, 128))
        return cudaErrorInvalidValue;
    const int items = plan.nseg ? plan.nsink * plan.nseg + plan.ntiles - plan.nsink : plan.ntiles;
    e = launch_plain(dkdv_tc_kernel<D, LENS>, dim3(a.Hk, a.B, items), dim3(kThreads), KvLayout<D>::BYTES, stream, a, plan, mq, mk, mv, mg);
    if (e == cudaSuccess)
        e = launch_plain(dq_tc_kernel<D, LENS>, dim3(a.Hq, a.B, (a.T + 127) / 128), dim3(kThreads), QLayout<D>::BYTES, stream, a, mq, mk,
                         mv, mg);
    if (e == cudaSuccess && plan.nseg && plan.nsink)
        e = launch_plain(sink_sum_kernel<D>, dim3(plan.nsink * 16, a.Hk, a.B), dim3(256), 0, stream, a, plan);
    return e;
}

}  // namespace

size_t swa_bwd_tc_partial_floats(const SwaArgs &a, int num_sms)
{
    const KvPlan p = plan_kv(a, num_sms);
    return p.nseg ? (size_t)a.B * a.Hk * p.nsink * p.nseg * 256 * a.d : 0;
}

cudaError_t launch_swa_bwd_tc(const SwaArgs &a, float *part, int num_sms, cudaStream_t stream)
{
    if (a.lens) return a.d == 128 ? impl<128, true>(a, part, num_sms, stream) : impl<64, true>(a, part, num_sms, stream);
    return a.d == 128 ? impl<128, false>(a, part, num_sms, stream) : impl<64, false>(a, part, num_sms, stream);
}

}  // namespace gdn2
