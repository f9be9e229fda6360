// win_delta.cu -- D_i of the rows at the first kExactDelta positions, for windowed
// attention's backward: D_i = sum_j P_ij dP_ij, P = 2^(c S - L log2 e), dP = dO V^T.
//
// Everywhere else D_i = sum_d dO_id O_id with the stored O, whose rounding to bf16 puts an
// error of up to 2^-8 sum_d |dO_id O_id| into every dS_ij / P_ij of the row.  |O| falls with the root of
// the keys a row sees, and a short sequence's gradients are dominated by its first rows:
// dQ's error was 1.6 times that of an fp32 computation rounded once at N = 101 (1.55 at
// 227), with these rows exact it is 1.4, which is what dS as a bf16 operand leaves.  128
// positions are what one tile of keys serves; behind them the share fades slowly (with that
// root), it does not end.
//
// A CTA has 32 rows of a query head and up to 128 keys: a warp has 16 rows and 32 keys, mma.sync
// (16 rows x 8 keys x 16 columns) on 64-column panels in shared memory, two at a time.
// Bound by its latency (about 7 us at D = 128 with cold caches, under the profiler), most of it
// beside the dQ kernel's start, which is launched as its dependent: one CTA a head with 16 rows x
// 128 keys a warp made the two kernels together 1.8 us slower (B3 H6/2 N1531 D80: 29.4 us, now 27.6).
#include "fa_internal.h"
#include "launch.cuh"
#include "sm100_ptx.cuh"
#include "win.cuh"
#include <algorithm>

namespace fa {
namespace {

constexpr int kKeys = kExactDelta;  // the rows see no later key
constexpr int kRows = 32;           // rows of a CTA
constexpr int kThreads = 256;
// a 64-column panel of Q, dO, K and V; two of them in shared memory at once
constexpr int kRowTile = kRows * 128, kKeyTile = kKeys * 128, kPanel = 2 * kRowTile + 2 * kKeyTile;
constexpr int kPanels = 2;
constexpr int kAlloc = kPanels * kPanel;
static_assert(kKeys == 128, "eight warps: two groups of 16 rows, four of 32 keys");

__global__ void __launch_bounds__(kThreads) win_delta_kernel(BwdArgs a, int parts) {
    launch_dependents();
    extern __shared__ __align__(128) uint8_t tiles[];  // 16-byte chunk c of row r at c ^ (r % 8)
    __shared__ float sums[kKeys / 32][kRows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row_group = warp & 1, key_group = warp >> 1;
    const int bh = blockIdx.x / parts, kv_bh = bh / a.H * a.win.Hkv + bh % a.H / (a.H / a.win.Hkv);
    const int off = a.win.Nk - a.N;  // position of row 0
    const int row0 = blockIdx.x % parts * kRows, rows = min(min(a.N, kExactDelta - off) - row0, kRows);  // >= 1
    const int keys = off + row0 + rows;  // the keys that the CTA's rows can see
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + ((size_t)bh * a.N + row0) * a.D;
    const __nv_bfloat16 *dO = static_cast<const __nv_bfloat16 *>(a.dO) + ((size_t)bh * a.N + row0) * a.D;
    const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(a.k) + (size_t)kv_bh * a.win.Nk * a.D;
    const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v) + (size_t)kv_bh * a.win.Nk * a.D;
    // one panel's tile; columns past D and rows past `n` are zeros
    auto load = [&](uint32_t to, const __nv_bfloat16 *from, int tile_rows, int n, int c0) {
        for (int x = threadIdx.x; x < tile_rows * 8; x += kThreads) {
            const int r = x >> 3, c = x & 7;
            const bool in = r < n && c0 + 8 * c < a.D;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + r * 128 + ((c ^ (r & 7)) << 4)),
                         "l"(from + (in ? (size_t)r * a.D + c0 + 8 * c : 0)), "r"(in ? 16 : 0)
                         : "memory");
        }
    };
    // fragments of S and dP: [16-key block][keys 0-7, 8-15]; element 2 r + e: row g + 8 r, key 2 tq + e
    float s[2][2][4], dp[2][2][4];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[b][h][e] = dp[b][h][e] = 0.f;
    // ldmatrix addresses: lane l gives row (l % 8) of matrix l / 8.
    //   rows as A: (rows 0-7, cols 0-7), (rows 8-15, cols 0-7), (rows 0-7, cols 8-15), (rows 8-15, cols 8-15)
    //   keys as B: (keys 0-7, cols 0-7), (keys 0-7, cols 8-15), (keys 8-15, ...) x 2
    const int mi = lane >> 3, mr = lane & 7;
    const uint32_t a_row = 16 * row_group + mr + (mi & 1) * 8, a_chunk = mi >> 1;
    const uint32_t b_row = 32 * key_group + mr + (mi >> 1) * 8, b_chunk = mi & 1;
    const uint32_t base = smem_u32(tiles);
    const bool busy = 32 * key_group < keys;  // some row sees a key of this warp's
    for (int c0 = 0; c0 < a.D; c0 += 64 * kPanels) {
        __syncthreads();  // the panels before have been read
#pragma unroll
        for (int p = 0; p < kPanels; ++p) {
            const uint32_t at = base + p * kPanel;
            const int c = c0 + 64 * p;
            if (c >= a.D) break;
            load(at, q, kRows, rows, c);
            load(at + kRowTile, dO, kRows, rows, c);
            load(at + 2 * kRowTile, k, kKeys, keys, c);
            load(at + 2 * kRowTile + kKeyTile, v, kKeys, keys, c);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        if (!busy) continue;
#pragma unroll
        for (int p = 0; p < kPanels; ++p) {
            if (c0 + 64 * p >= a.D) break;
            const uint32_t qs = base + p * kPanel, ks = qs + 2 * kRowTile;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                uint32_t qf[4], gf[4];
                ldsm4(qf, qs + a_row * 128 + (((2 * kk + a_chunk) ^ mr) << 4));
                ldsm4(gf, qs + kRowTile + a_row * 128 + (((2 * kk + a_chunk) ^ mr) << 4));
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    uint32_t kf[4], vf[4];
                    ldsm4(kf, ks + (16 * b + b_row) * 128 + (((2 * kk + b_chunk) ^ mr) << 4));
                    ldsm4(vf, ks + kKeyTile + (16 * b + b_row) * 128 + (((2 * kk + b_chunk) ^ mr) << 4));
                    mma16816(s[b][0], qf, kf[0], kf[1]);
                    mma16816(s[b][1], qf, kf[2], kf[3]);
                    mma16816(dp[b][0], gf, vf[0], vf[1]);
                    mma16816(dp[b][1], gf, vf[2], vf[3]);
                }
            }
        }
    }
    const int g = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = 16 * row_group + g + 8 * r, p = off + row0 + row;
        const float l2 = row < rows ? a.lse[(size_t)bh * a.N + row0 + row] * 1.4426950408889634f : 0.f;
        float delta = 0.f;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int key = 32 * key_group + 16 * b + 8 * h + 2 * tq + e;
                    if (key <= p && (key < a.win.sinks || key > p - a.win.window))
                        delta = fmaf(ex2_approx(fmaf(s[b][h][2 * r + e], a.scale_log2, -l2)), dp[b][h][2 * r + e], delta);
                }
        delta += __shfl_xor_sync(0xffffffffu, delta, 1);
        delta += __shfl_xor_sync(0xffffffffu, delta, 2);
        if (tq == 0) sums[key_group][row] = delta;
    }
    __syncthreads();
    if ((int)threadIdx.x < rows) {
        float delta = 0.f;
#pragma unroll
        for (int x = 0; x < kKeys / 32; ++x) delta += sums[x][threadIdx.x];
        a.delta[(size_t)bh * a.N + row0 + threadIdx.x] = delta;
    }
}

}  // namespace

cudaError_t launch_win_delta(const BwdArgs &a, cudaStream_t s) {
    static std::atomic<unsigned long long> allowed{0};
    cudaError_t e = allow_smem((const void *)win_delta_kernel, kAlloc, allowed);
    if (e != cudaSuccess) return e;
    const int rows = std::min(a.N, kExactDelta - (a.win.Nk - a.N)), parts = (rows + kRows - 1) / kRows;
    return launch_behind(win_delta_kernel, dim3(a.B * a.H * parts), kThreads, kAlloc, false, 1, s, a, parts);
}

}  // namespace fa
