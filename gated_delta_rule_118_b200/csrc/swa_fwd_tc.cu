// swa_fwd_tc.cu -- windowed attention forward for bf16 on the tensor cores.
//
// A CTA takes 256 query rows of a head at a time, as two tiles of 128 rows that share
// every key and value tile of 128 keys, and works in blocks of 64 keys.  One warp loads
// tiles by TMA (two-stage rings of K and of V); for each query tile a warp issues the
// products and a warpgroup does the softmax, one row per thread:
//   S = Q K^T            operands in shared memory, S in tensor memory
//   P = exp2(S - m)      read from tensor memory, written back over S as bf16
//   O += P V             A operand straight from tensor memory
// Each query tile has two score buffers: the scores of block u + 1 are computed while
// block u is in its softmax.  What bounds the kernel is the chain of hand-overs (a product's
// completion takes about 335 cycles to be seen, a barrier about 100): with one buffer of
// 128 keys a tile, kernels with a quarter of the products and no exponentials took 70 % of
// the time.  Two tiles x two buffers keep four chains in flight.
// 16 heads of 128, window 2048, 4 sinks: 1 x 4096 82 to 85 us, 1 x 16384 302 to 316 us (about
// 840 TFLOP/s, the tensor pipe active 40 % of the time); heads of 64: 75 and 283 us; 8192
// causal, 16 heads of 128 over 4, 270 us (1017 TFLOP/s).
//
// CTAs are persistent: a CTA that finishes asks the hardware for a block that has not
// started (cluster launch control) and runs it, so the next rows' loads and first scores
// overlap the last rows' writes.
//
// A row's reference m need not be its maximum: it stands in the exponent of every term
// and in the final sum alike, P is rounded relative to its own size, and fp32 and bf16
// reach to 2^127.  So a row takes its reference from the first tile it sees and keeps it;
// later tiles whose keys are all visible are exponentiated without looking for a maximum
// first (which was a quarter of the softmax), and only a tile whose sum comes out at 2^60
// or more, or not finite, is taken again with a new reference (and O rescaled in tensor
// memory).  Tiles with masked keys look for their maximum, and raise the reference when a
// row outgrows it by more than 2^8.
// P is rounded to bf16 for the product (at most 2^-8 relative, as the operand of
// a bf16 tensor core has to be); the row sum adds the unrounded values in fp32.
#include <cuda.h>

#include "launch.h"
#include "sm100.cuh"
#include "swa_common.cuh"
#include "tc_common.cuh"

namespace gdn2 {
namespace {

using namespace swa;
using namespace sm100;

constexpr int kThreads = 384;  // two softmax warpgroups, then the issuing warps
constexpr int kTma = 8, kNext = 9, kMma = 10;  // kMma + t issues the products of query tile t
// 384 threads launch with 168 registers each; a softmax row keeps 64 scores and their
// exponentials in registers, the issuing warps need fewer: 2 x 128 x 200 + 128 x 104 = 384 x 168.
constexpr int kRegsSoftmax = 200, kRegsIssue = 104;
constexpr float kMaxGrowth = 8.f;         // log2
constexpr float kMaxSum = 0x1p60f;        // of a tile exponentiated by an old reference

template <int D>
struct Layout {
    static constexpr int TILE = 128 * D * 2;       // bytes of a 128-row tile, boxes of 64 channels
    static constexpr int Q = 0, K = 2 * TILE, V = 4 * TILE, BAR = 6 * TILE;
    static constexpr int NEXT = BAR + 256;         // answer of the launch control
    static constexpr int SLOT = NEXT + 16;
    static constexpr int BYTES = SLOT + 16 + 1024;
    static constexpr uint32_t TM_O = 256;          // scores of tile t at 128 t (two buffers of 64), then the outputs
};

// mbarriers
enum { Q_FULL, Q_EMPTY, K_FULL, K_EMPTY = K_FULL + 2, V_FULL = K_EMPTY + 2, V_EMPTY = V_FULL + 2,
       S_FULL = V_EMPTY + 2,      // [tile][buffer]
       P_FULL = S_FULL + 4,       // [tile][buffer], one arrival of each softmax warp
       O_DONE = P_FULL + 4,       // [tile]: a product P V is in O
       O_LAST = O_DONE + 2,       // [tile]: the last one of these rows is
       N_FULL = O_LAST + 2, N_EMPTY, DRAINED,
       V_TAIL = DRAINED + 2,      // a V tile that holds padding has landed
       NBAR };
// released by the issuing warps of both query tiles
__host__ __device__ constexpr bool both_tiles(int i)
{
    return i == Q_EMPTY || i == K_EMPTY || i == K_EMPTY + 1 || i == V_EMPTY || i == V_EMPTY + 1;
}
constexpr int kReaders = 12;      // warps that read the launch control's answer

// The 256 query rows of one block of the grid: the rows that see most keys first, of all
// heads and sequences, so that the short ones fill the gaps at the end.
struct Work {
    int i0, h, b, n;
    __device__ __forceinline__ Work(const SwaArgs &a, int x, int y, int z)
        : i0((gridDim.z - 1 - z) * 256), h(x), b(y), n(seq_len(a, y)) {}
    __device__ __forceinline__ KeyTiles tiles(const SwaArgs &a) const
    {
        const int off = a.Tk - a.T;
        return KeyTiles(off + i0, off + min(i0 + 256, n) - 1, a.window, a.sinks, 128);
    }
};

// The blocks of 64 keys that one query tile visits, and those all of whose keys all of
// its rows see.
struct Visits {
    int w0, ns, last;        // visited: [w0, last], and below ns
    int wf, nf, lf;          // full: [wf, lf], and below nf up to lf
    __device__ __forceinline__ Visits(const SwaArgs &a, int i0, int n)
    {
        const int p0 = a.Tk - a.T + i0, p1 = a.Tk - a.T + min(i0 + 128, n) - 1;
        w0 = (p0 - a.window + 1 > 0 ? p0 - a.window + 1 : 0) >> 6;
        ns = (a.sinks + 63) >> 6;
        last = i0 < n ? p1 >> 6 : -1;  // -1: no row of this tile holds a token
        wf = p0 + 127 - a.window < 0 ? 0 : ((p0 + 127 - a.window) >> 6) + 1;
        nf = a.sinks >> 6;
        lf = (p0 - 63) >> 6;
    }
    __device__ __forceinline__ bool operator()(int j) const { return j <= last && (j >= w0 || j < ns); }
    __device__ __forceinline__ bool full(int j) const { return j <= lf && (j >= wf || j < nf); }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
fwd_tc_kernel(const __grid_constant__ SwaArgs a, const __grid_constant__ CUtensorMap mq,
              const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv)
{
    using L = Layout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::BAR);
    uint8_t *answer = sm + L::NEXT;
    uint32_t *slot = reinterpret_cast<uint32_t *>(sm + L::SLOT);
    static_assert(NBAR * 8 <= 256, "room for the barriers");
    if (tid == 0) {
        for (int i = 0; i < NBAR; ++i)
            mbar_init(bar + i, i >= P_FULL && i < P_FULL + 4 ? 4 : i == N_EMPTY ? kReaders : both_tiles(i) ? 2 : 1);
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
    int bx = blockIdx.x, by = blockIdx.y, bz = blockIdx.z;
    uint32_t nph = 0;
    // the next block for this warp (false: none, or a wait gave up)
    auto advance = [&](bool ok) {
        ok = __all_sync(~0u, ok && mbar_wait(bar + N_FULL, nph, a.err));
        if (!ok) return false;
        nph ^= 1;
        const bool more = next_cta(answer, bx, by, bz);
        fence_proxy_async_smem();  // the next answer is written by the async proxy
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + N_EMPTY);
        return more;
    };

    if (warp >= 8) {
        setmaxnreg_dec<kRegsIssue>();
        if (warp == kNext) {
            bool more = true;
            for (uint32_t eph = 1; more; eph ^= 1) {
                bool ok = mbar_wait(bar + N_EMPTY, eph, a.err);
                ok = __all_sync(~0u, ok);
                if (ok && elect_one()) {
                    mbar_arrive_expect_tx(bar + N_FULL, 16);
                    next_cta_request(answer, bar + N_FULL);
                }
                __syncwarp();
                more = advance(ok);
            }
        } else if (warp == kTma) {
            uint32_t kt_count = 0, qph = 0;  // tiles asked for; both rings advance together
            uint32_t tph = 0;
            bool ok = true, more = true;
            while (more) {
                const Work w(a, bx, by, bz);
                if (w.i0 < w.n) {
                    const int hk = w.h / (a.Hq / a.Hk);
                    const KeyTiles kt = w.tiles(a);
                    ok = __all_sync(~0u, mbar_wait(bar + Q_EMPTY, qph ^ 1, a.err));
                    qph ^= 1;
                    if (!ok) break;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(bar + Q_FULL, 2 * L::TILE);
                        for (int t = 0; t < 2; ++t)
                            for (int x = 0; x < D / 64; ++x)
                                tma_load_4d(sm + L::Q + t * L::TILE + x * 16384, &mq, bar + Q_FULL, x * 64, w.h,
                                            w.i0 + t * 128, w.b);
                    }
                    __syncwarp();
                    for (int c = 0; ok && c < kt.count(); ++c, ++kt_count) {
                        const int s = kt_count & 1, j0 = kt.tile(c) * 128;
                        const uint32_t ph = ((kt_count >> 1) & 1) ^ 1;
                        ok = __all_sync(~0u, mbar_wait(bar + K_EMPTY + s, ph, a.err));
                        if (ok && elect_one()) {
                            mbar_arrive_expect_tx(bar + K_FULL + s, L::TILE);
                            for (int x = 0; x < D / 64; ++x)
                                tma_load_4d(sm + L::K + s * L::TILE + x * 16384, &mk, bar + K_FULL + s, x * 64, hk, j0, w.b);
                        }
                        __syncwarp();
                        if (!ok) break;
                        ok = __all_sync(~0u, mbar_wait(bar + V_EMPTY + s, ph, a.err));
                        // (the last tile of a block's, if any)
                        const int keys = a.Tk - a.T + w.n;  // behind them is padding
                        const bool tail = w.n < a.T && j0 + 128 > keys;
                        uint64_t *landed = bar + (tail ? V_TAIL : V_FULL + s);
                        if (elect_one()) {
                            // asked for also after a failed wait: both rings stay in step for the drain below
                            mbar_arrive_expect_tx(landed, L::TILE);
                            for (int x = 0; x < D / 64; ++x)
                                tma_load_4d(sm + L::V + s * L::TILE + x * 16384, &mv, landed, x * 64, hk, j0, w.b);
                        }
                        __syncwarp();
                        if (tail) {
                            ok = __all_sync(~0u, mbar_wait(landed, tph, a.err)) && ok;
                            tph ^= 1;
                            zero_rows<D>(sm + L::V + s * L::TILE, keys - j0);
                            if (lane == 0) mbar_arrive(bar + V_FULL + s);
                        }
                    }
                }
                more = advance(ok);
            }
            // every copy has landed before the CTA ends, also when another role gave up
            for (uint32_t c = kt_count < 2 ? 0 : kt_count - 2; c < kt_count; ++c) {
                mbar_wait(bar + K_FULL + (c & 1), (c >> 1) & 1, a.err);
                mbar_wait(bar + V_FULL + (c & 1), (c >> 1) & 1, a.err);
            }
            if (qph || kt_count) mbar_wait(bar + Q_FULL, qph ^ 1, a.err);
        } else if (warp >= kMma) {
            // the whole warp walks the loop and one lane issues: the descriptors stay in
            // uniform registers (computed in one lane's registers every product cost about
            // 100 cycles of issue)
            const int t = warp - kMma;
            const uint32_t id_s = idesc_bf16(128, 64, 0, 0), id_o = idesc_bf16(128, D, 0, 1);
            constexpr uint32_t STEP = L::TILE >> 4;  // descriptor units (16 bytes) of a tile
            const uint64_t dq = smem_desc(sbase + L::Q, 16, 1024, kSw128) + t * STEP, dk = smem_desc(sbase + L::K, 16, 1024, kSw128);
            const uint64_t dv = smem_desc(sbase + L::V, 16384, 1024, kSw128);
            const uint32_t ts = tmem + t * 128, to = tmem + L::TM_O + t * D;
            uint32_t kc = 0, vc = 0, qph = 0;        // tiles consumed, blocks of the grid with work
            uint32_t ns = 0, np = 0;                 // score blocks and P V products issued
            auto commit = [&](int which) {
                if (elect_one()) umma_commit(bar + which);
                __syncwarp();
            };
            bool ok = true, more = true;
            while (more) {
                const Work w(a, bx, by, bz);
                if (w.i0 < w.n) {
                    const Visits v(a, w.i0 + t * 128, w.n);
                    const KeyTiles kt = w.tiles(a);
                    const int nu = 2 * kt.count();
                    uint32_t acc = 0;
                    ok = __all_sync(~0u, mbar_wait(bar + Q_FULL, qph, a.err));
                    qph ^= 1;
                    for (int u = 0; ok && u <= nu; ++u) {
                        const uint32_t hf = u & 1;
                        if (u < nu) {  // scores of block u
                            const uint32_t s = kc & 1;
                            if (!hf) ok = __all_sync(~0u, mbar_wait(bar + K_FULL + s, (kc >> 1) & 1, a.err));
                            if (!ok) break;
                            if (v(kt.tile(u >> 1) * 2 + hf)) {
                                // (over P of the block before last, whose product was issued
                                // before: products run in order)
                                tc_fence_after();
                                if (elect_one()) {
#pragma unroll
                                    for (int ks = 0; ks < D / 16; ++ks) {
                                        const uint32_t o = (ks >> 2) * 1024 + (ks & 3) * 2;
                                        umma_bf16(ts + (ns & 1) * 64, dq + o, dk + (s * STEP + hf * 512 + o), id_s, ks > 0);
                                    }
                                    umma_commit(bar + S_FULL + 2 * t + (ns & 1));
                                }
                                __syncwarp();
                                ++ns;
                            }
                            if (hf) {
                                commit(K_EMPTY + s);
                                ++kc;
                            }
                            if (u == nu - 1) commit(Q_EMPTY);
                        }
                        if (u > 0) {   // outputs of block u - 1
                            const uint32_t s = vc & 1, bf = np & 1;
                            const int j = kt.tile((u - 1) >> 1) * 2 + (hf ^ 1);
                            if (hf) ok = mbar_wait(bar + V_FULL + s, (vc >> 1) & 1, a.err);
                            if (v(j)) {
                                ok = ok && mbar_wait(bar + P_FULL + 2 * t + bf, (np >> 1) & 1, a.err);
                                ok = __all_sync(~0u, ok);
                                tc_fence_after();
                                if (ok && elect_one()) {
#pragma unroll
                                    for (int ks = 0; ks < 4; ++ks)
                                        umma_bf16_ts(to, ts + bf * 64 + ks * 8, dv + (s * STEP + (hf ^ 1) * 512 + ks * 128), id_o,
                                                     acc | (ks > 0));
                                    umma_commit(bar + O_DONE + t);
                                    if (j == v.last) umma_commit(bar + O_LAST + t);
                                }
                                __syncwarp();
                                acc = 1;
                                ++np;
                            }
                            ok = __all_sync(~0u, ok);
                            if (!ok) break;
                            if (!hf) {
                                commit(V_EMPTY + s);
                                ++vc;
                            }
                        }
                    }
                }
                more = advance(ok);
            }
            commit(DRAINED + t);  // no product is in flight when the tensor memory is freed
            mbar_wait(bar + DRAINED + t, 0, a.err);
        }
    } else {
        setmaxnreg_inc<kRegsSoftmax>();
        const int t = warp >> 2, r = tid & 127;
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t to = lane_base + L::TM_O + t * D;
        const float sc = a.scale * kLog2E;
        uint32_t ns = 0, lph = 0;  // blocks of scores this tile has taken, phase of O_LAST
        bool ok = true, more = true;
        while (more) {
            const Work w(a, bx, by, bz);
            const int row = w.i0 + t * 128 + r, p = a.Tk - a.T + row;
            const bool live = row < w.n;  // (what the rows behind hold must not decide for the warp)
            float m = -INFINITY, l = 0.f;
            bool started = false;
            if (w.i0 < w.n) {
                const Visits visits(a, w.i0 + t * 128, w.n);
                const KeyTiles kt = w.tiles(a);
                const int nu = 2 * kt.count();
                for (int u = 0; u < nu; ++u) {
                    const int j = kt.tile(u >> 1) * 2 + (u & 1);
                    if (!visits(j)) continue;
                    const uint32_t bf = ns & 1, ts = lane_base + t * 128 + bf * 64;
                    ok = __all_sync(~0u, mbar_wait(bar + S_FULL + 2 * t + bf, (ns >> 1) & 1, a.err));
                    if (!ok) break;
                    tc_fence_after();
                    float s[64], sum[4];
                    uint32_t v[32];
                    auto take_scores = [&] {
                        tmem_ld32(ts, *reinterpret_cast<float(*)[32]>(s));
                        tmem_ld32(ts + 32, *reinterpret_cast<float(*)[32]>(s + 32));
                        tmem_ld_wait(s);
                    };
                    auto exponentials = [&](float ms) {
                        sum[0] = sum[1] = sum[2] = sum[3] = 0.f;
#pragma unroll
                        for (int x = 0; x < 64; x += 2) {
                            const float e0 = ex2_approx(fmaf(s[x], sc, -ms)), e1 = ex2_approx(fmaf(s[x + 1], sc, -ms));
                            sum[x & 2] += e0;
                            sum[(x & 2) + 1] += e1;
                            const __nv_bfloat162 e = __floats2bfloat162_rn(e0, e1);
                            v[x / 2] = *reinterpret_cast<const uint32_t *>(&e);
                        }
                    };
                    const bool full = visits.full(j);
                    bool careful = !full || __any_sync(~0u, live && m == -INFINITY);
                    take_scores();
                    if (__builtin_expect(!careful, 1)) {
                        exponentials(m);
                        careful = __any_sync(~0u, live && !((sum[0] + sum[1]) + (sum[2] + sum[3]) < kMaxSum));
                        if (__builtin_expect(careful, 0)) take_scores();
                    }
                    if (__builtin_expect(careful, 0)) {
                        if (!full) {
                            const int j0 = j * 64, hi = p - j0, lo = p - a.window + 1 - j0, sk = a.sinks - j0;
#pragma unroll
                            for (int x = 0; x < 64; ++x) s[x] = x <= hi && (x >= lo || x < sk) ? s[x] : -INFINITY;
                        }
                        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                        for (int x = 4; x < 64; x += 4)
#pragma unroll
                            for (int y = 0; y < 4; ++y) mx[y] = fmaxf(mx[y], s[x + y]);
                        const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
                        const bool grow = mt > m + kMaxGrowth;  // also the first finite score of the row
                        if (__any_sync(~0u, grow)) {
                            const float f = grow ? ex2_approx(m - mt) : 1.f;
                            if (grow) m = mt;
                            l *= f;
                            if (started) {
                                // rescale O, once the product before this block is in it.  (The one
                                // before that was complete when these scores were, so the parity is
                                // unambiguous.)
                                ok = __all_sync(~0u, mbar_wait(bar + O_DONE + t, (ns - 1) & 1, a.err));
                                if (!ok) break;
                                tc_fence_after();
                                for (int x = 0; x < D; x += 16) {
                                    float o[16];
                                    tmem_ld16(to + x, o);
                                    tmem_ld_wait(o);
                                    uint32_t g[16];
#pragma unroll
                                    for (int y = 0; y < 16; ++y) g[y] = __float_as_uint(o[y] * f);
                                    tmem_st16(to + x, g);
                                }
                            }
                        }
                        exponentials(m == -INFINITY ? 0.f : m);
                    }
                    started = true;
                    tmem_st32(ts, v);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar + P_FULL + 2 * t + bf);
                    ++ns;
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                }
            }
            // write the row; rows that are not finite are formed again from memory
            if (started && ok) {
                ok = mbar_wait(bar + O_LAST + t, lph, a.err);
                lph ^= 1;
                ok = __all_sync(~0u, ok);
                tc_fence_after();
            }
            if (ok) {
                const bool inside = row < a.T;
                const float inv = l == 0.f ? 0.f : 1.f / l;
                bf16 *dst = static_cast<bf16 *>(a.out) + (((long long)w.b * a.T + row) * a.Hq + w.h) * D;
                bool bad = false;
#pragma unroll
                for (int x = 0; x < D; x += 32) {
                    float o[32];
                    if (started) {
                        tmem_ld32(to + x, o);
                        tmem_ld_wait(o);
                    }
#pragma unroll
                    for (int y = 0; y < 32; ++y) {
                        o[y] = live && started ? o[y] * inv : 0.f;
                        bad |= !isfinite(o[y]);
                    }
                    if (inside)
#pragma unroll
                        for (int y = 0; y < 32; y += 8) *reinterpret_cast<uint4 *>(dst + x + y) = pack8(o + y);
                }
                tc_fence_before();  // O is read before the next rows' products overwrite it
                if (a.lse && inside)
                    a.lse[((long long)w.b * a.Hq + w.h) * a.T + row] = !live || l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
                unsigned todo = __ballot_sync(~0u, bad);
                __syncwarp();
                while (todo) {
                    const int r0 = __ffs(todo) - 1;
                    todo &= todo - 1;
                    row_forward<bf16, D>(a, w.b, w.h, row - lane + r0);
                }
            }
            more = advance(ok);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D>
cudaError_t impl(const SwaArgs &a, cudaStream_t stream)
{
    using L = Layout<D>;
    auto kern = fwd_tc_kernel<D>;
    static std::atomic<unsigned long long> smem_set{0};
    cudaError_t e = ensure_smem_limit(kern, L::BYTES, smem_set);
    if (e != cudaSuccess) return e;
    CUtensorMap mq, mk, mv;
    if (!make_rows_map(&mq, a.q, D, a.Hq, a.T, a.B, a.qs, 128) || !make_rows_map(&mk, a.k, D, a.Hk, a.Tk, a.B, a.ks, 128) ||
        !make_rows_map(&mv, a.v, D, a.Hk, a.Tk, a.B, a.vs, 128))
        return cudaErrorInvalidValue;
    return launch_plain(kern, dim3(a.Hq, a.B, (a.T + 255) / 256), dim3(kThreads), L::BYTES, stream, a, mq, mk, mv);
}

}  // namespace

cudaError_t launch_swa_fwd_tc(const SwaArgs &a, cudaStream_t stream)
{
    return a.d == 128 ? impl<128>(a, stream) : impl<64>(a, stream);
}

}  // namespace gdn2
