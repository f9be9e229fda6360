// win_sinks.cu -- what the rows far behind a few sinks (at most 16) add to the sinks' dK
// and dV, for D = 64.  Those rows see the sinks and none of the other keys of the
// sinks' 128-key tile, so win_dkdv.cu would spend a full tile's work on them.
//
//   S^T = K_s Q^T,  P^T = 2^(c S^T - L log2 e),  dV_s += P^T dO,
//   dP^T = V_s dO^T,  dS^T = P^T (dP^T - D),     dK_s += dS^T Q  (times scale at the end)
//
// Bound by HBM: every row of Q and dO is read once for 16 keys, 4 x 16 multiply-adds a
// byte pair, far below the tensor cores' rate at that bandwidth, so the products are
// 16 keys x 8 rows x 16 columns mma.sync (a tcgen05 product has 64 keys at least).
//   warp 4     TMA producer: 128-row tiles of Q and dO into a ring
//   warps 0-3  16 rows of each half of every tile, dK_s and dV_s in registers; joined at the
//              end (8 warps of two CTAs an SM; twice as many spilled and took 95 us
//              instead of 50 for 32 heads of 32768 rows: 5.3 TB/s)
// For D = 64 only: a warp keeps dK_s and dV_s (16 keys x 64 columns each) in 64 registers a lane
// of the 168 that two CTAs leave; twice the columns would have to be dealt to twice the warps.
// A CTA takes one chunk of a key head's rows (win_key_item) and writes an fp32 partial,
// which sink_sum_kernel adds in a fixed order.
#include "fa_internal.h"
#include "launch.cuh"
#include "sm100_ptx.cuh"
#include "win.cuh"

namespace fa {
namespace {

constexpr int kD = 64;
constexpr int kRows = 128;  // rows per tile, as the tensor maps of win_dkdv.cu have them
constexpr int kWarps = 4;
constexpr int kHalves = kRows / (16 * kWarps);
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kStages = 3;
constexpr int kTile = kRows * kD * 2;
constexpr int kKeyBytes = kFewSinks * kD * 2;
constexpr int kKeyOff = kStages * 2 * kTile;  // K_s, V_s
constexpr int kBarOff = kKeyOff + 2 * kKeyBytes;
constexpr int kAlloc = kBarOff + 2 * kStages * 8 + 1024;
static_assert(kFewSinks == 16, "the rows of one product");
static_assert(kWarps * 2 * kFewSinks * kD * 4 <= kStages * 2 * kTile, "the join goes over the ring");
static_assert(2 * (kAlloc + 1024) <= 233472, "two CTAs on an SM");

enum : int { kSiteEmpty = 261, kSiteFull, kSiteDrain };

__global__ void __launch_bounds__(kThreads, 2)
    win_sinks_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_do, BwdArgs a,
                     float *part_dk, float *part_dv) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kBarOff);
    uint64_t *empty = full + kStages;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const WinKeyItem w = win_key_item(a, blockIdx.x, 128, kRows);
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kWarps);
        }
        fence_mbarrier_init();
    }
    // K_s and V_s (16-byte chunk c of row r at c ^ (r % 8)); columns past D and rows past the last key are zeros
    for (int e = threadIdx.x; e < 2 * kFewSinks * 8; e += kThreads) {
        const int c = e & 7, r = (e >> 3) % kFewSinks, which = e / (8 * kFewSinks);
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (r < a.win.Nk && 8 * c < a.D)
            x = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(which ? a.v : a.k) +
                                                 ((size_t)w.bh * a.win.Nk + r) * a.D + 8 * c);
        *reinterpret_cast<uint4 *>(smem + kKeyOff + which * kKeyBytes + r * 128 + ((c ^ (r & 7)) << 4)) = x;
    }
    __syncthreads();
    launch_dependent_wait();  // D comes from the dQ kernel

    float dk[kD / 8][4], dv[kD / 8][4];
#pragma unroll
    for (int i = 0; i < kD / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) dk[i][e] = dv[i][e] = 0.f;
    const int g = lane >> 2, tq = lane & 3;  // fragment row (key g and g + 8), column pair
    bool ok = true;

    if (warp == kWarps) {
        if (lane == 0) {
            tma_prefetch_desc(&tmap_q);
            tma_prefetch_desc(&tmap_do);
            WinRowWalk at(a, w);
            for (int i = 0; i < w.n; ++i, at.next()) {
                const int s = i % kStages, round = i / kStages;
                if (!mbar_wait(&empty[s], (round & 1) ^ 1, a.status, kSiteEmpty)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(&full[s], 2 * kTile);
                tma_load_3d(smem + s * 2 * kTile, &tmap_q, &full[s], 0, w.rows.first + at.h * kRows, at.slice);
                tma_load_3d(smem + s * 2 * kTile + kTile, &tmap_do, &full[s], 0, w.rows.first + at.h * kRows, at.slice);
            }
            // the loads of the last rounds have landed before the CTA reuses or leaves its shared memory
            for (int i = max(0, w.n - kStages); i < w.n && ok; ++i)
                mbar_wait(&full[i % kStages], (i / kStages) & 1, a.status, kSiteDrain);
        }
    } else {
        constexpr float kLog2e = 1.4426950408889634f;
        // L and D of this lane's four rows of each half: 2 tq, 2 tq + 1, and 8 behind each
        float l[kHalves][4], d[kHalves][4];
        auto load_stats = [&](const WinRowWalk &at) {
#pragma unroll
            for (int u = 0; u < 4 * kHalves; ++u) {
                const int row = w.rows.first + at.h * kRows + 64 * (u >> 2) + 16 * warp + 8 * (u >> 1 & 1) + 2 * tq + (u & 1);
                const bool valid = row < a.N;
                const size_t x = (size_t)at.slice * a.N + (valid ? row : 0);
                l[u >> 2][u & 3] = valid ? a.lse[x] : INFINITY;
                d[u >> 2][u & 3] = valid ? a.delta[x] : 0.f;
            }
        };
        // ldmatrix addresses: lane l gives row (l % 8) of matrix l / 8.
        //   K_s, V_s (keys x columns): (keys 0-7, cols 0-7), (keys 8-15, cols 0-7), (keys 0-7, cols 8-15), (8-15, 8-15)
        //   Q, dO (rows x columns): (rows 0-7, cols 0-7), (rows 0-7, cols 8-15), (rows 8-15, ...) x 2
        //   the same transposed: (rows 0-7, cols 0-7), (rows 8-15, cols 0-7), (rows 0-7, cols 8-15), ...
        const int mi = lane >> 3, mr = lane & 7;
        const uint32_t a_row = mr + (mi & 1) * 8, a_chunk = mi >> 1;
        const uint32_t b_row = 16 * warp + mr + (mi >> 1) * 8, b_chunk = mi & 1;
        const uint32_t t_row = 16 * warp + mr + (mi & 1) * 8, t_chunk = mi >> 1;
        const uint32_t base = smem_u32(smem), keys = base + kKeyOff;
        // out = A B^T over the 64 columns: keys x this warp's 16 rows
        auto scores = [&](float (&sc)[2][4], uint32_t a_s, uint32_t b_s) {
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[0][e] = sc[1][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < kD / 16; ++kk) {
                uint32_t af[4], bf[4];
                ldsm4(af, a_s + a_row * 128 + (((2 * kk + a_chunk) ^ mr) << 4));
                ldsm4(bf, b_s + b_row * 128 + (((2 * kk + b_chunk) ^ mr) << 4));
                mma16816(sc[0], af, bf[0], bf[1]);
                mma16816(sc[1], af, bf[2], bf[3]);
            }
        };
        auto add_product = [&](float (&acc)[kD / 8][4], const uint32_t (&pf)[4], uint32_t b_s) {
#pragma unroll
            for (int dd = 0; dd < kD / 16; ++dd) {
                uint32_t bf[4];
                ldsm4t(bf, b_s + t_row * 128 + (((2 * dd + t_chunk) ^ mr) << 4));
                mma16816(acc[2 * dd], pf, bf[0], bf[1]);
                mma16816(acc[2 * dd + 1], pf, bf[2], bf[3]);
            }
        };
        WinRowWalk at(a, w);
        if (w.n > 0) load_stats(at);
        for (int i = 0; i < w.n; ++i) {
            const int s = i % kStages;
            float ln[kHalves][4], dn[kHalves][4];  // this tile's; the next tile's are on their way meanwhile
#pragma unroll
            for (int u = 0; u < 4 * kHalves; ++u) ln[u >> 2][u & 3] = l[u >> 2][u & 3], dn[u >> 2][u & 3] = d[u >> 2][u & 3];
            at.next();
            if (i + 1 < w.n) load_stats(at);
            ok = mbar_wait(&full[s], (i / kStages) & 1, a.status, kSiteFull);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
                const uint32_t qs = base + s * 2 * kTile + h * 64 * 128, dos = qs + kTile;
                float st[2][4], dp[2][4];
                scores(st, keys, qs);
                scores(dp, keys + kKeyBytes, dos);
                uint32_t pf[4], dsf[4];
                // fragment element: key g + 8 r, rows 8 n + 2 tq and the one behind it.  Keys past the sinks: P = dS = 0
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        float p[2], ds[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const bool seen = g + 8 * r < a.win.sinks;
                            p[e] = seen ? ex2_approx(fmaf(st[n][2 * r + e], a.scale_log2, -ln[h][2 * n + e] * kLog2e)) : 0.f;
                            ds[e] = seen ? p[e] * (dp[n][2 * r + e] - dn[h][2 * n + e]) : 0.f;
                        }
                        // the products' operands, rounded to bf16 as in win_dkdv.cu
                        pf[2 * n + r] = pack_bf16x2(p[0], p[1]);
                        dsf[2 * n + r] = pack_bf16x2(ds[0], ds[1]);
                    }
                __syncwarp();
                add_product(dv, pf, dos);
                add_product(dk, dsf, qs);
            }
            warp_arrive(&empty[s]);
        }
    }
    // join the warps' sums over the ring (every tile has landed and been read), in order
    __syncthreads();
    float *jo = reinterpret_cast<float *>(smem);  // [2][kWarps][16][64]
    if (warp < kWarps) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int c = 0; c < kD / 8; ++c) {
                float *at = jo + (warp * kFewSinks + g + 8 * r) * kD + 8 * c + 2 * tq;
                *reinterpret_cast<float2 *>(at) = make_float2(dk[c][2 * r], dk[c][2 * r + 1]);
                *reinterpret_cast<float2 *>(at + kWarps * kFewSinks * kD) = make_float2(dv[c][2 * r], dv[c][2 * r + 1]);
            }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * kFewSinks * kD; e += kThreads) {
        const int which = e / (kFewSinks * kD), in = e % (kFewSinks * kD), r = in / kD, c = in % kD;
        float s = 0.f;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) s += jo[(which * kWarps + x) * kFewSinks * kD + in];
        if (c < a.D) (which ? part_dv : part_dk)[((size_t)w.part * 128 + r) * a.D + c] = which ? s : s * a.scale;
    }
}

}  // namespace

cudaError_t launch_win_sinks(const BwdArgs &a, const CUtensorMap &tq, const CUtensorMap &tdo, float *part_dk, float *part_dv,
                             cudaStream_t s) {
    static std::atomic<unsigned long long> allowed{0};
    cudaError_t e = allow_smem((const void *)win_sinks_kernel, kAlloc, allowed);
    if (e != cudaSuccess) return e;
    return launch_behind(win_sinks_kernel, dim3(a.B * a.win.Hkv * a.win.chunks), kThreads, kAlloc, true, 1, s, tq, tdo, a,
                         part_dk, part_dv);
}

}  // namespace fa
