// swa_fwd_tc.cu -- windowed attention forward for bf16 on the tensor cores.
//
// One CTA per 256 query rows of a head, as two tiles of 128 rows that share every
// key and value tile of 128 keys.  Warp 9 loads tiles by TMA (two-stage rings of K
// and of V), warp 8 issues the products, and a warpgroup per query tile does the
// softmax, one row per thread:
//   S = Q K^T            operands in shared memory, S in tensor memory
//   P = exp2(S - m)      read from tensor memory, written back over S as bf16
//   O += P V             A operand straight from tensor memory
// While one tile is in its softmax the tensor core works on the other tile, so the
// pair runs at the slower of the two.  Bound by that softmax/tensor alternation:
// a 128 x 128 score tile is 16384 exponentials, 1024 cycles of the SM's special
// function units, as many as its two products take on the tensor core.
//
// The running maximum is only raised (and O rescaled in tensor memory) when a row
// outgrows its reference by more than 2^8: with the reference in the exponent of
// every term and in the final sum alike, any reference gives the same result as
// long as nothing overflows, and P is rounded relative to its own size.
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

constexpr int kThreads = 320;
constexpr float kMaxGrowth = 8.f;  // log2

template <int D>
struct Layout {
    static constexpr int TILE = 128 * D * 2;       // bytes of a 128-row tile, boxes of 64 channels
    static constexpr int Q = 0, K = 2 * TILE, V = 4 * TILE, BAR = 6 * TILE;
    static constexpr int NBAR = 1 + 8 + 6 + 1;
    static constexpr int SLOT = BAR + 8 * NBAR;
    static constexpr int BYTES = SLOT + 16 + 1024;
    static constexpr uint32_t TM_O = 256;          // S tiles at 0 and 128, O tiles at 256 and 256 + D
};

// The key tiles that one query tile visits.
struct Tile {
    int p0, p1, w0, st, last;
    __device__ __forceinline__ Tile(const SwaArgs &a, int i0, int n)
    {
        p0 = a.Tk - a.T + i0;
        p1 = a.Tk - a.T + min(i0 + 128, n) - 1;
        const int lo = p0 - a.window + 1 > 0 ? p0 - a.window + 1 : 0;
        w0 = lo >> 7;
        st = (a.sinks + 127) >> 7;
        last = p1 >= p0 ? p1 >> 7 : -1;            // -1: no row of this tile holds a token
    }
    __device__ __forceinline__ bool visits(int j) const { return j <= last && (j >= w0 || j < st); }
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
    const int i0 = (gridDim.x - 1 - blockIdx.x) * 256, h = blockIdx.y, b = blockIdx.z;  // longest rows first
    const int n = seq_len(a, b), hk = h / (a.Hq / a.Hk);
    bf16 *out = static_cast<bf16 *>(a.out) + (((long long)b * a.T + i0) * a.Hq + h) * D;
    const long long ost = (long long)a.Hq * D;
    float *lse = a.lse ? a.lse + ((long long)b * a.Hq + h) * a.T + i0 : nullptr;
    if (i0 >= n) {  // padding only
        const int rows = min(256, a.T - i0);
        for (int c = tid; c < rows * (D / 8); c += kThreads)
            *reinterpret_cast<uint4 *>(out + c / (D / 8) * ost + c % (D / 8) * 8) = make_uint4(0, 0, 0, 0);
        if (lse)
            for (int r = tid; r < rows; r += kThreads) lse[r] = -INFINITY;
        return;
    }
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::BAR);
    uint64_t *q_full = bar, *k_full = bar + 1, *k_empty = bar + 3, *v_full = bar + 5, *v_empty = bar + 7;
    uint64_t *s_full = bar + 9, *p_full = bar + 11, *o_full = bar + 13, *drained = bar + 15;
    uint32_t *slot = reinterpret_cast<uint32_t *>(sm + L::SLOT);
    if (tid == 0) {
        for (int i = 0; i < L::NBAR; ++i) mbar_init(bar + i, (bar + i == p_full || bar + i == p_full + 1) ? 128 : 1);
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot;
    const int off = a.Tk - a.T;
    const KeyTiles kt(off + i0, off + min(i0 + 256, n) - 1, a.window, a.sinks, 128);
    const int ntiles = kt.count();
    const uint32_t sbase = smem_u32(sm);

    if (warp == 9) {
        if (lane == 0) {
            mbar_arrive_expect_tx(q_full, 2 * L::TILE);
            for (int t = 0; t < 2; ++t)
                for (int x = 0; x < D / 64; ++x)
                    tma_load_4d(sm + L::Q + t * L::TILE + x * 16384, &mq, q_full, x * 64, h, i0 + t * 128, b);
            int nk = 0, nv = 0;  // tiles asked for
            for (int c = 0; c < ntiles; ++c) {
                const int s = c & 1, j0 = kt.tile(c) * 128;
                const uint32_t ph = ((c >> 1) & 1) ^ 1;
                if (!mbar_wait(k_empty + s, ph, a.err)) break;
                nk = c + 1;
                mbar_arrive_expect_tx(k_full + s, L::TILE);
                for (int x = 0; x < D / 64; ++x)
                    tma_load_4d(sm + L::K + s * L::TILE + x * 16384, &mk, k_full + s, x * 64, hk, j0, b);
                if (!mbar_wait(v_empty + s, ph, a.err)) break;
                nv = c + 1;
                mbar_arrive_expect_tx(v_full + s, L::TILE);
                for (int x = 0; x < D / 64; ++x)
                    tma_load_4d(sm + L::V + s * L::TILE + x * 16384, &mv, v_full + s, x * 64, hk, j0, b);
            }
            // every copy has landed before the CTA ends, also when another role gave up
            for (int c = max(nk - 2, 0); c < nk; ++c) mbar_wait(k_full + (c & 1), (c >> 1) & 1, a.err);
            for (int c = max(nv - 2, 0); c < nv; ++c) mbar_wait(v_full + (c & 1), (c >> 1) & 1, a.err);
        }
    } else if (warp == 8) {
        if (lane == 0) {
            const Tile t0(a, i0, n), t1(a, i0 + 128, n);
            const uint32_t id_s = idesc_bf16(128, 128, 0, 0), id_o = idesc_bf16(128, D, 0, 1);
            uint32_t pph[2] = {0, 0}, acc[2] = {0, 0};
            auto scores = [&](int t, int s) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t o = (ks >> 2) * 16384 + (ks & 3) * 32;
                    umma_bf16(tmem + t * 128, smem_desc(sbase + L::Q + t * L::TILE + o, 16, 1024, kSw128),
                              smem_desc(sbase + L::K + s * L::TILE + o, 16, 1024, kSw128), id_s, ks > 0);
                }
                umma_commit(s_full + t);
            };
            bool ok = mbar_wait(q_full, 0, a.err);
            ok = ok && mbar_wait(k_full, 0, a.err);
            if (ok) {
                tc_fence_after();
                if (t0.visits(kt.tile(0))) scores(0, 0);
                if (t1.visits(kt.tile(0))) scores(1, 0);
                umma_commit(k_empty);
            }
            for (int c = 0; ok && c < ntiles; ++c) {
                const int s = c & 1, j = kt.tile(c), jn = c + 1 < ntiles ? kt.tile(c + 1) : -1;
                const uint32_t ph = (c >> 1) & 1;
                ok = mbar_wait(v_full + s, ph, a.err);
                if (ok && jn >= 0) ok = mbar_wait(k_full + (s ^ 1), ((c + 1) >> 1) & 1, a.err);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const Tile &tt = t ? t1 : t0;
                    if (ok && tt.visits(j)) {
                        ok = mbar_wait(p_full + t, pph[t], a.err);
                        pph[t] ^= 1;
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            umma_bf16_ts(tmem + L::TM_O + t * D, tmem + t * 128 + ks * 8,
                                         smem_desc(sbase + L::V + s * L::TILE + ks * 2048, 16384, 1024, kSw128), id_o,
                                         acc[t] | (ks > 0));
                        acc[t] = 1;
                        if (j == tt.last) umma_commit(o_full + t);
                    }
                    if (ok && jn >= 0 && tt.visits(jn)) scores(t, s ^ 1);
                }
                if (!ok) break;
                umma_commit(v_empty + s);
                if (jn >= 0) umma_commit(k_empty + (s ^ 1));
            }
            umma_commit(drained);  // no product is in flight when the tensor memory is freed
            mbar_wait(drained, 0, a.err);
        }
    } else {
        const int t = warp >> 2, r = tid & 127, row = t * 128 + r;  // row within the pair
        const Tile tt(a, i0 + t * 128, n);
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t ts = lane_base + t * 128, to = lane_base + L::TM_O + t * D;
        const int p = tt.p0 + r;
        const float sc = a.scale * kLog2E;
        float m = -INFINITY, l = 0.f;
        uint32_t sph = 0;
        bool ok = true, started = false;
        for (int c = 0; c < ntiles; ++c) {
            const int j = kt.tile(c), j0 = j * 128;
            if (!tt.visits(j)) continue;
            ok = mbar_wait(s_full + t, sph, a.err);
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            sph ^= 1;
            tc_fence_after();
            float s[128];
#pragma unroll
            for (int x = 0; x < 4; ++x) tmem_ld32(ts + x * 32, *reinterpret_cast<float(*)[32]>(s + x * 32));
            tmem_ld_wait();
            if (!tile_full(tt.p0, tt.p0 + 127, j0, j0 + 128, a.window, a.sinks)) {
                const int hi = p - j0, lo = p - a.window + 1 - j0, sk = a.sinks - j0;
#pragma unroll
                for (int x = 0; x < 128; ++x) s[x] = x <= hi && (x >= lo || x < sk) ? s[x] : -INFINITY;
            }
            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int x = 4; x < 128; x += 4)
#pragma unroll
                for (int y = 0; y < 4; ++y) mx[y] = fmaxf(mx[y], s[x + y]);
            const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
            const bool grow = mt > m + kMaxGrowth;  // also the first finite score of the row
            if (__any_sync(~0u, grow)) {
                const float f = grow ? ex2_approx(m - mt) : 1.f;
                if (grow) m = mt;
                l *= f;
                if (started) {  // there is an O to rescale
                    for (int x = 0; x < D; x += 32) {
                        float o[32];
                        tmem_ld32(to + x, o);
                        tmem_ld_wait();
                        uint32_t u[32];
#pragma unroll
                        for (int y = 0; y < 32; ++y) u[y] = __float_as_uint(o[y] * f);
                        tmem_st32(to + x, u);
                    }
                }
            }
            started = true;
            const float ms = m == -INFINITY ? 0.f : m;
            float sum[4] = {};
#pragma unroll
            for (int x = 0; x < 128; x += 64) {
                uint32_t u[32];
#pragma unroll
                for (int y = 0; y < 64; y += 2) {
                    const float e0 = ex2_approx(fmaf(s[x + y], sc, -ms)), e1 = ex2_approx(fmaf(s[x + y + 1], sc, -ms));
                    sum[y & 2] += e0;
                    sum[(y & 2) + 1] += e1;
                    const __nv_bfloat162 e = __floats2bfloat162_rn(e0, e1);
                    u[y / 2] = *reinterpret_cast<const uint32_t *>(&e);
                }
                tmem_st32(ts + x / 2, u);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(p_full + t);
        }
        // write the row; rows that are not finite are formed again from memory
        if (started && ok) {
            ok = mbar_wait(o_full + t, 0, a.err);
            ok = __all_sync(~0u, ok);
            tc_fence_after();
        }
        const bool live = row + i0 < n, inside = row + i0 < a.T;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        bf16 *dst = out + row * ost;
        bool bad = false;
        for (int x = 0; x < D; x += 32) {
            float o[32] = {};
            if (started) {
                tmem_ld32(to + x, o);
                tmem_ld_wait();
            }
#pragma unroll
            for (int y = 0; y < 32; ++y) {
                o[y] = live ? o[y] * inv : 0.f;
                bad |= !isfinite(o[y]);
            }
            if (inside)
#pragma unroll
                for (int y = 0; y < 32; y += 8) *reinterpret_cast<uint4 *>(dst + x + y) = pack8(o + y);
        }
        if (lse && inside) lse[row] = !live || l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        unsigned todo = __ballot_sync(~0u, bad && live && ok);
        __syncwarp();
        while (todo) {
            const int r0 = __ffs(todo) - 1;
            todo &= todo - 1;
            row_forward<bf16, D>(a, b, h, i0 + row - lane + r0);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
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
    kern<<<dim3((a.T + 255) / 256, a.Hq, a.B), kThreads, L::BYTES, stream>>>(a, mq, mk, mv);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_swa_fwd_tc(const SwaArgs &a, cudaStream_t stream)
{
    return a.d == 128 ? impl<128>(a, stream) : impl<64>(a, stream);
}

}  // namespace gdn2
