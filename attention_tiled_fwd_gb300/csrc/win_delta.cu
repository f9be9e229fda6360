// win_delta.cu -- D_i of the rows at the first kExactDelta positions, for windowed
// attention's backward: D_i = sum_j P_ij dP_ij, P = 2^(c S - L log2 e), dP = dO V^T.
//
// Everywhere else D_i = sum_d dO_id O_id with the stored O, whose rounding to bf16 puts an
// error of |dO||O| 2^-9 or so into every dS_ij / P_ij of the row.  |O| falls with the root of
// the keys a row sees, so a short sequence's gradients, which the first rows dominate,
// carried as much error from it as from half of dS's own rounding (dQ's error 1.6 times
// that of an fp32 computation rounded once at N = 101, 1.55 at 227; with these rows
// exact 1.4, which is what dS as a bf16 operand leaves).
//
// One CTA a query head: 128 rows x 128 keys, 8 warps of 16 rows, mma.sync (16 rows x 8 keys
// x 16 columns) on 64-column panels in shared memory.  Bound by its latency (9 us at D = 128, most of
// it behind the dQ kernel's start, which is launched as its dependent).
#include "fa_internal.h"
#include "launch.cuh"
#include "sm100_ptx.cuh"
#include "win.cuh"

namespace fa {
namespace {

constexpr int kRows = kExactDelta;  // rows, and keys: the rows see no later key
constexpr int kWarps = kRows / 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = kRows * 64 * 2;  // one 64-column panel of Q, dO, K or V
constexpr int kAlloc = 4 * kTile;
static_assert(kRows == 128, "eight warps, eight blocks of 16 keys");

__global__ void __launch_bounds__(kThreads) win_delta_kernel(BwdArgs a) {
    launch_dependents();
    extern __shared__ __align__(128) uint8_t tiles[];  // Q, dO, K, V: 16-byte chunk c of row r at c ^ (r % 8)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int bh = blockIdx.x, kv_bh = bh / a.H * a.win.Hkv + bh % a.H / (a.H / a.win.Hkv);
    const int off = a.win.Nk - a.N;  // position of row 0
    const int rows = min(a.N, kRows - off), keys = min(a.win.Nk, kRows);
    const __nv_bfloat16 *src[4] = {static_cast<const __nv_bfloat16 *>(a.q) + (size_t)bh * a.N * a.D,
                                   static_cast<const __nv_bfloat16 *>(a.dO) + (size_t)bh * a.N * a.D,
                                   static_cast<const __nv_bfloat16 *>(a.k) + (size_t)kv_bh * a.win.Nk * a.D,
                                   static_cast<const __nv_bfloat16 *>(a.v) + (size_t)kv_bh * a.win.Nk * a.D};
    // fragments of S and dP: [16-key block][keys 0-7, 8-15]; element 2 r + e: row g + 8 r, key 2 tq + e
    float s[kRows / 16][2][4], dp[kRows / 16][2][4];
#pragma unroll
    for (int b = 0; b < kRows / 16; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[b][h][e] = dp[b][h][e] = 0.f;
    const int last = off + 16 * warp + 15;  // this warp's last position
    // ldmatrix addresses: lane l gives row (l % 8) of matrix l / 8.
    //   rows as A: (rows 0-7, cols 0-7), (rows 8-15, cols 0-7), (rows 0-7, cols 8-15), (rows 8-15, cols 8-15)
    //   keys as B: (keys 0-7, cols 0-7), (keys 0-7, cols 8-15), (keys 8-15, ...) x 2
    const int mi = lane >> 3, mr = lane & 7;
    const uint32_t a_row = 16 * warp + mr + (mi & 1) * 8, a_chunk = mi >> 1, b_row = mr + (mi >> 1) * 8, b_chunk = mi & 1;
    const uint32_t base = smem_u32(tiles);
    for (int c0 = 0; c0 < a.D; c0 += 64) {
        __syncthreads();  // the panel before has been read
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < kRows * 8 / kThreads; ++i) {
                const int x = threadIdx.x + i * kThreads, r = x >> 3, c = x & 7;
                const bool in = r < (t < 2 ? rows : keys) && c0 + 8 * c < a.D;  // else zeros
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(base + t * kTile + r * 128 + ((c ^ (r & 7)) << 4)),
                             "l"(src[t] + (in ? (size_t)r * a.D + c0 + 8 * c : 0)), "r"(in ? 16 : 0)
                             : "memory");
            }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            uint32_t qf[4], gf[4];
            ldsm4(qf, base + a_row * 128 + (((2 * kk + a_chunk) ^ mr) << 4));
            ldsm4(gf, base + kTile + a_row * 128 + (((2 * kk + a_chunk) ^ mr) << 4));
#pragma unroll
            for (int b = 0; b < kRows / 16; ++b) {
                if (16 * b > last) continue;  // no row of this warp sees those keys
                uint32_t kf[4], vf[4];
                ldsm4(kf, base + 2 * kTile + (16 * b + b_row) * 128 + (((2 * kk + b_chunk) ^ mr) << 4));
                ldsm4(vf, base + 3 * kTile + (16 * b + b_row) * 128 + (((2 * kk + b_chunk) ^ mr) << 4));
                mma16816(s[b][0], qf, kf[0], kf[1]);
                mma16816(s[b][1], qf, kf[2], kf[3]);
                mma16816(dp[b][0], gf, vf[0], vf[1]);
                mma16816(dp[b][1], gf, vf[2], vf[3]);
            }
        }
    }
    const int g = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = 16 * warp + g + 8 * r, p = off + row;
        const size_t at = (size_t)bh * a.N + row;
        const float l2 = row < rows ? a.lse[at] * 1.4426950408889634f : 0.f;
        float delta = 0.f;
#pragma unroll
        for (int b = 0; b < kRows / 16; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int key = 16 * b + 8 * h + 2 * tq + e;
                    if (key <= p && (key < a.win.sinks || key > p - a.win.window))
                        delta = fmaf(ex2_approx(fmaf(s[b][h][2 * r + e], a.scale_log2, -l2)), dp[b][h][2 * r + e], delta);
                }
        delta += __shfl_xor_sync(0xffffffffu, delta, 1);
        delta += __shfl_xor_sync(0xffffffffu, delta, 2);
        if (row < rows && tq == 0) a.delta[at] = delta;
    }
}

}  // namespace

cudaError_t launch_win_delta(const BwdArgs &a, cudaStream_t s) {
    static std::atomic<unsigned long long> allowed{0};
    cudaError_t e = allow_smem((const void *)win_delta_kernel, kAlloc, allowed);
    if (e != cudaSuccess) return e;
    return launch_behind(win_delta_kernel, dim3(a.B * a.H), kThreads, kAlloc, false, 1, s, a);
}

}  // namespace fa
