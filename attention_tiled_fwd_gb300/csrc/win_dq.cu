// win_dq.cu -- dQ of windowed attention for D = 128 (D = 64 runs win_dq_k128.cu, wider
// heads bwd_dq.cu).  Per
// 128-row query tile, over the key tiles that its rows see (key_span):
//
//   D_i = sum_d dO_id O_id (written out),
//   S = Q K_j^T,  P = 2^(c S - L log2 e),  dP = dO V_j^T,  dS = P (dP - D),
//   dQ += dS K_j  (times scale at the end)
//
// Products, TMEM layout and roles are bwd_dq.cu's at D = 128: 64-key tiles, S and
// dP double-buffered, Q as the TMEM operand of S, dS as that of dQ; warp 0 TMA
// producer, warp 1 issuer A (S, dP), warp 2 issuer B (dQ), warps 3-10 compute, a
// thread owning one row and half of each tile's keys.
//
// A window of 1024 gives a tile 18 key tiles, 10 us of products beside 4 us of fixed
// cost per CTA, so the grid is one CTA per SM that walks tiles.  The next tile's Q
// and O share one buffer (both are consumed at a tile's start), dO has two; once
// the compute warps have seen a tile's last S they copy the next tile's Q into TMEM
// and only then write dQ, so issuer A is two key tiles ahead when they come back.
// Bound by the chain S, dP -> compute -> dQ of its 64-key tiles: B2 H16/4 N4096 window
// 1024: 103 us with win_delta.cu's kernel before it, 878 TFLOP/s of the visible pairs
// (three products each).
#include "fa_internal.h"
#include "launch.cuh"
#include "sm100_ptx.cuh"
#include "win.cuh"
#include <cmath>

namespace fa {
namespace {

constexpr int kD = 128;
constexpr int kBM = 128;        // queries per item (TMEM lanes)
constexpr int kBN = kDqKRows;   // keys per tile
constexpr int kComputeWG = 2;   // one 32-key half of every tile each
constexpr int kHalf = kBN / kComputeWG;
constexpr int kFirstComputeWarp = 3;
constexpr int kComputeWarps = 4 * kComputeWG;
constexpr int kThreads = 32 * (kFirstComputeWarp + kComputeWarps);
constexpr int kPanels = kD / 64;
constexpr int kSlots = 6;       // K_j / V_j ring

enum : int { kSiteQ = 241, kSiteSlotEmpty, kSiteSlotFull, kSiteSFull, kSiteDsFull, kSiteDq, kSiteFinal, kSiteDrain,
             kSiteDqDone, kSiteQt, kSiteAcc, kSiteQEmpty, kSiteDoEmpty };

struct WinDqSmem {
    static constexpr int kQBytes = kBM * kD * 2;
    static constexpr int kTileBytes = kBN * kD * 2;
    static constexpr int kQOff = 0, kOOff = kQBytes, kDoOff = 2 * kQBytes;  // Q, O, dO[2]
    static constexpr int kSlotOff = 4 * kQBytes;
    static constexpr int kDeltaOff = kSlotOff + kSlots * kTileBytes;  // [kComputeWG][kBM] partial sums
    static constexpr int kBarOff = kDeltaOff + kComputeWG * kBM * 4;
    // qo_full, qo_empty, do_full[2], do_empty[2], slot_full/empty[kSlots], s_full[2], ds_full[2], dq_done[2], qt_ready,
    // acc_full, acc_free, final, a_final
    static constexpr int kNumBars = 6 + 2 * kSlots + 6 + 5;
    static constexpr int kTmemHolderOff = kBarOff + kNumBars * 8;
    static constexpr int kAlloc = kTmemHolderOff + 16 + 1024;
    static_assert(kAlloc <= 232448, "shared memory budget");
};

__global__ void __launch_bounds__(kThreads, 1)
    win_dq_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                  const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_do,
                  const __grid_constant__ CUtensorMap tmap_o, const __grid_constant__ CUtensorMap tmap_dq, BwdArgs a,
                  int n_items) {
    using L = WinDqSmem;
    constexpr uint32_t kTmemCols = 512;
    // S[b] = [64b, +64), dP[b] = [128 + 64b, +64), dQ = [256, 384), dS[b] = [384 + 32b, +32), Q = [448, 512)
    constexpr uint32_t kColDP = 128, kColDQ = 256, kColDS = 384, kColQ = 448;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *q_s = smem + L::kQOff, *o_s = smem + L::kOOff;
    uint8_t *slots = smem + L::kSlotOff;
    float *delta_s = reinterpret_cast<float *>(smem + L::kDeltaOff);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBarOff);
    uint64_t *qo_full = bars;                  // item n's Q and O landed
    uint64_t *qo_empty = qo_full + 1;          // every compute warp has read them
    uint64_t *do_full = qo_empty + 1;          // [2]: item n's dO landed in buffer n % 2
    uint64_t *do_empty = do_full + 2;          // [2]: its dQ, staged over dO, has been stored
    uint64_t *slot_full = do_empty + 2;
    uint64_t *slot_empty = slot_full + kSlots;
    uint64_t *s_full = slot_empty + kSlots;    // [2]: S and dP of step t complete (steps counted across items)
    uint64_t *ds_full = s_full + 2;            // [2]: dS of step t written (and S, dP read)
    uint64_t *dq_done = ds_full + 2;           // [2]: dQ product of step t complete
    uint64_t *qt_ready = dq_done + 2;          // item n's Q is in TMEM
    uint64_t *acc_full = qt_ready + 1;         // item n's dQ is complete
    uint64_t *acc_free = acc_full + 1;         // every compute warp has read it
    uint64_t *final_bar = acc_free + 1;
    uint64_t *a_final = final_bar + 1;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + L::kTmemHolderOff);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(qo_full, 1);
        mbar_init(qo_empty, kComputeWarps);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&do_full[b], 1);
            mbar_init(&do_empty[b], 1);
            mbar_init(&s_full[b], 1);
            mbar_init(&ds_full[b], kComputeWarps);
            mbar_init(&dq_done[b], 1);
        }
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(&slot_full[s], 1);
            mbar_init(&slot_empty[s], 1);
        }
        mbar_init(qt_ready, kComputeWarps);
        mbar_init(acc_full, 1);
        mbar_init(acc_free, kComputeWarps);
        mbar_init(final_bar, 1);
        mbar_init(a_final, 1);
        fence_mbarrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    launch_dependents();  // the dK/dV kernel of the same call fills the SMs as they come free
    const uint32_t tmem = *tmem_holder;

    // Every role walks the same items: persistent_work_index deals them, n counts this CTA's.
    if (warp == 0) {
        if (lane == 0) {
            tma_prefetch_desc(&tmap_q);
            tma_prefetch_desc(&tmap_k);
            tma_prefetch_desc(&tmap_v);
            tma_prefetch_desc(&tmap_do);
            tma_prefetch_desc(&tmap_o);
            int last_round[kSlots];
#pragma unroll
            for (int s = 0; s < kSlots; ++s) last_round[s] = -1;
            bool ok = true;
            int n = 0, t = 0, n_do = 0;
            for (int k = 0; ok && k * (int)gridDim.x < n_items; ++k) {
                const int x = persistent_work_index(k, n_items);
                if (x < 0) continue;
                const WinRowItem w = win_row_item(a, x, kBM, kBN);
                if (n >= 1 && !(ok = mbar_wait(qo_empty, (n - 1) & 1, a.status, kSiteQEmpty))) break;
                mbar_arrive_expect_tx(qo_full, 2 * L::kQBytes);
#pragma unroll
                for (int p = 0; p < kPanels; ++p) {
                    tma_load_3d(q_s + p * (kBM * 128), &tmap_q, qo_full, p * 64, w.row0, w.bh);
                    tma_load_3d(o_s + p * (kBM * 128), &tmap_o, qo_full, p * 64, w.row0, w.bh);
                }
                ++n;
                const int buf = n_do & 1;
                if (n_do >= 2 && !(ok = mbar_wait(&do_empty[buf], ((n_do >> 1) - 1) & 1, a.status, kSiteDoEmpty))) break;
                uint8_t *do_s = smem + L::kDoOff + buf * L::kQBytes;
                mbar_arrive_expect_tx(&do_full[buf], L::kQBytes);
#pragma unroll
                for (int p = 0; p < kPanels; ++p)
                    tma_load_3d(do_s + p * (kBM * 128), &tmap_do, &do_full[buf], p * 64, w.row0, w.bh);
                ++n_do;
                for (int j = 0; ok && j < w.span.n; ++j, ++t) {
                    const int key0 = w.span.key0(j, kBN);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // K_j, V_j
                        const int idx = 2 * t + h, slot = idx % kSlots, round = idx / kSlots;
                        if (!(ok = mbar_wait(&slot_empty[slot], (round & 1) ^ 1, a.status, kSiteSlotEmpty))) break;
                        uint8_t *dst = slots + slot * L::kTileBytes;
                        mbar_arrive_expect_tx(&slot_full[slot], L::kTileBytes);
#pragma unroll
                        for (int p = 0; p < kPanels; ++p)
                            tma_load_3d(dst + p * (kBN * 128), h ? &tmap_v : &tmap_k, &slot_full[slot], p * 64, key0,
                                        w.kv_bh);
#pragma unroll
                        for (int s = 0; s < kSlots; ++s)
                            if (s == slot) last_round[s] = round;
                    }
                }
            }
            // Drain: never leave the CTA with a TMA write still in flight.
#pragma unroll
            for (int s = 0; s < kSlots; ++s)
                if (last_round[s] >= 0) mbar_wait(&slot_full[s], last_round[s] & 1, a.status, kSiteDrain);
            if (n >= 1) mbar_wait(qo_full, (n - 1) & 1, a.status, kSiteDrain);
            if (n_do >= 2) mbar_wait(&do_full[n_do & 1], ((n_do - 2) >> 1) & 1, a.status, kSiteDrain);
            if (n_do >= 1) mbar_wait(&do_full[(n_do - 1) & 1], ((n_do - 1) >> 1) & 1, a.status, kSiteDrain);
        }
        __syncwarp();
    } else if (warp == 1) {
        // Issuer A: S = Q K_j^T (Q from TMEM) and dP = dO V_j^T into buffer t % 2.
        constexpr uint32_t idesc_sq = idesc_bf16_f32(kBM, kBN, false, false);
        const uint32_t slot_addr = smem_u32(slots);
        const bool leader = elect_one();
        bool ok = true;
        int n = 0, t = 0;
        for (int k = 0; ok && k * (int)gridDim.x < n_items; ++k) {
            const int x = persistent_work_index(k, n_items);
            if (x < 0) continue;
            const WinRowItem w = win_row_item(a, x, kBM, kBN);
            if (!(ok = warp_wait(&do_full[n & 1], (n >> 1) & 1, a.status, kSiteQ))) break;
            if (!(ok = warp_wait(qt_ready, n & 1, a.status, kSiteQt))) break;
            const uint64_t do_desc = sdesc_sw128(smem_u32(smem + L::kDoOff + (n & 1) * L::kQBytes), 16, 1024);
            ++n;
            for (int j = 0; j < w.span.n; ++j, ++t) {
                const uint32_t b = t & 1;
                const int k_slot = (2 * t) % kSlots, v_slot = (2 * t + 1) % kSlots;
                // S[b], dP[b] last held step t-2, which the compute warps have finished with
                if (t >= 2 && !(ok = warp_wait(&ds_full[b], ((t - 2) >> 1) & 1, a.status, kSiteDsFull))) break;
                if (!(ok = warp_wait(&slot_full[k_slot], (2 * t / kSlots) & 1, a.status, kSiteSlotFull))) break;
                if (!(ok = warp_wait(&slot_full[v_slot], ((2 * t + 1) / kSlots) & 1, a.status, kSiteSlotFull))) break;
                tc_fence_after();
                const uint64_t k_desc = sdesc_sw128(slot_addr + k_slot * L::kTileBytes, 16, 1024);
                const uint64_t v_desc = sdesc_sw128(slot_addr + v_slot * L::kTileBytes, 16, 1024);
                if (leader) {
#pragma unroll
                    for (int ks = 0; ks < kD / 16; ++ks)
                        mma_ts(tmem + 64 * b, tmem + kColQ + ks * 8,
                               sdesc_add(k_desc, (ks >> 2) * (kBN * 128) + (ks & 3) * 32), idesc_sq, ks > 0);
#pragma unroll
                    for (int ks = 0; ks < kD / 16; ++ks)
                        mma_ss(tmem + kColDP + 64 * b, sdesc_add(do_desc, (ks >> 2) * (kBM * 128) + (ks & 3) * 32),
                               sdesc_add(v_desc, (ks >> 2) * (kBN * 128) + (ks & 3) * 32), idesc_sq, ks > 0);
                    mma_commit(&s_full[b]);
                    mma_commit(&slot_empty[v_slot]);  // V_j is no longer needed
                }
                __syncwarp();
            }
        }
        if (leader) mma_commit(a_final);
        __syncwarp();
        warp_wait(a_final, 0, a.status, kSiteFinal);
    } else if (warp == 2) {
        // Issuer B: dQ += dS K_j.
        constexpr uint32_t idesc_dq = idesc_bf16_f32(kBM, kD, false, true);
        const uint32_t slot_addr = smem_u32(slots);
        const bool leader = elect_one();
        bool ok = true;
        int n = 0, t = 0;
        for (int k = 0; ok && k * (int)gridDim.x < n_items; ++k) {
            const int x = persistent_work_index(k, n_items);
            if (x < 0) continue;
            const WinRowItem w = win_row_item(a, x, kBM, kBN);
            for (int j = 0; j < w.span.n; ++j, ++t) {
                const uint32_t b = t & 1;
                const int k_slot = (2 * t) % kSlots;
                const uint64_t kmn_desc = sdesc_sw128(slot_addr + k_slot * L::kTileBytes, kBN * 128, 1024);
                if (!(ok = warp_wait(&ds_full[b], (t >> 1) & 1, a.status, kSiteDsFull))) break;
                // the first product overwrites dQ, which the item before's epilogue reads
                if (j == 0 && n >= 1 && !(ok = warp_wait(acc_free, (n - 1) & 1, a.status, kSiteAcc))) break;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < kBN / 16; ++kk)
                        mma_ts(tmem + kColDQ, tmem + kColDS + 32 * b + kk * 8, sdesc_add(kmn_desc, kk * 2048), idesc_dq,
                               (j > 0 || kk > 0));
                    mma_commit(&dq_done[b]);
                    mma_commit(&slot_empty[k_slot]);  // S completed before dS was written
                }
                __syncwarp();
            }
            if (!ok) break;
            if (leader) mma_commit(acc_full);
            __syncwarp();
            ++n;
        }
        if (leader) mma_commit(final_bar);
        __syncwarp();
        warp_wait(final_bar, 0, a.status, kSiteFinal);
    } else {
        const int quarter = warp & 3;
        const int g = (warp - kFirstComputeWarp) >> 2;  // key half of every tile
        const int r = quarter * 32 + lane;
        const int sw = r & 7;
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        const uint64_t c2 = f2_pack(a.scale_log2, a.scale_log2);
        // a wait that ran out in one warp ends the loop in all of them: they meet at barrier 1, and none comes back
        // to it once one of them was not well (dead)
        bool dead = false;
        auto all_ok = [&](bool mine) {
            int go;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, 1, %2, p;\n\t"
                "selp.s32 %0, 1, 0, q;\n\t}"
                : "=r"(go)
                : "r"((int)mine), "r"(32 * kComputeWarps)
                : "memory");
            dead = go == 0;
            return go != 0;
        };
        // Item n's Q into TMEM as bf16 pairs, one 64-column panel per warpgroup (row r of a panel is 128 B at r * 128,
        // its 16-byte chunk c at c ^ (r % 8)); every S product of the item before has completed.
        auto copy_q = [&](int n) {
            bool got = mbar_wait(qo_full, n & 1, a.status, kSiteQ);
            if (!__all_sync(0xffffffffu, got)) return false;
            const uint8_t *panel = q_s + g * (kBM * 128) + r * 128;
            uint32_t v[32];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const uint4 u = *reinterpret_cast<const uint4 *>(panel + ((c ^ sw) << 4));
                v[4 * c] = u.x, v[4 * c + 1] = u.y, v[4 * c + 2] = u.z, v[4 * c + 3] = u.w;
            }
            tmem_st32(tmem + lane_base + kColQ + 32 * g, v);
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(qt_ready);
            return true;
        };
        // Item n's dQ (times the scale) through dO's buffer, which no product reads any more, as 128-byte-swizzled
        // panels of 128 rows (64 bf16 or 32 fp32 columns), 64 columns at a time; TMA stores clip rows past N and
        // columns past the caller's D.
        auto epilogue = [&](int n, const WinRowItem &w) {
            const bool got = mbar_wait(acc_full, n & 1, a.status, kSiteDq);
            if (!all_ok(got)) return false;
            tc_fence_after();
            uint8_t *stage = smem + L::kDoOff + (n & 1) * L::kQBytes;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t v[32];
                tmem_ld32(tmem + lane_base + kColDQ + 64 * h + 32 * g, v);
                tmem_wait_ld();
                if (h == 1) {
                    tc_fence_before();
                    warp_arrive(acc_free);
                    if (!a.grad_bf16) {  // the first half's store has read the area
                        if (threadIdx.x == 32 * kFirstComputeWarp) tma_store_wait_read();
                        asm volatile("bar.sync 1, %0;" ::"r"(32 * kComputeWarps) : "memory");
                    }
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * a.scale);
                if (a.grad_bf16) {
                    uint8_t *prow = stage + h * (kBM * 128) + r * 128;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        st_shared_v4(prow + (((4 * g + c) ^ sw) << 4),
                                     pack_bf16x2(__uint_as_float(v[8 * c + 0]), __uint_as_float(v[8 * c + 1])),
                                     pack_bf16x2(__uint_as_float(v[8 * c + 2]), __uint_as_float(v[8 * c + 3])),
                                     pack_bf16x2(__uint_as_float(v[8 * c + 4]), __uint_as_float(v[8 * c + 5])),
                                     pack_bf16x2(__uint_as_float(v[8 * c + 6]), __uint_as_float(v[8 * c + 7])));
                } else {
                    uint8_t *prow = stage + g * (kBM * 128) + r * 128;
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        st_shared_v4(prow + ((c ^ sw) << 4), v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
                }
                if (h == 1 || !a.grad_bf16) {
                    fence_proxy_async_smem();  // the staged panels are read by the TMA (async proxy)
                    asm volatile("bar.sync 1, %0;" ::"r"(32 * kComputeWarps) : "memory");
                    if (threadIdx.x == 32 * kFirstComputeWarp) {
                        const int pw = a.grad_bf16 ? 64 : 32;
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            const int col = (a.grad_bf16 ? 0 : 64 * h) + p * pw;
                            if (col < a.D) tma_store_3d(&tmap_dq, stage + p * (kBM * 128), col, w.row0, w.bh);
                        }
                        tma_store_commit();
                    }
                }
            }
            if (threadIdx.x == 32 * kFirstComputeWarp) {
                tma_store_wait_read();
                mbar_arrive(&do_empty[n & 1]);
            }
            return true;
        };

        bool ok = true;
        int n = 0, t = 0;
        WinRowItem prev{};
        for (int k = 0; ok && k * (int)gridDim.x < n_items; ++k) {
            const int x = persistent_work_index(k, n_items);
            if (x < 0) continue;
            const WinRowItem w = win_row_item(a, x, kBM, kBN);
            const int row = w.row0 + r;
            const bool valid = row < a.N;
            // P = 2^(S c - L log2 e); rows past the last get P = 0
            const float lse2 = valid ? a.lse[(size_t)w.bh * a.N + row] * 1.4426950408889634f : INFINITY;
            ok = copy_q(n);
            if (n > 0 && !(ok = all_ok(ok) && epilogue(n - 1, prev))) break;
            // D_i: warpgroup g sums columns [64g, 64g + 64); O's and dO's chunks sit at the same swizzled places
            float delta = 0.f;
            {
                const bool got = ok && mbar_wait(&do_full[n & 1], (n >> 1) & 1, a.status, kSiteQ);
                ok = __all_sync(0xffffffffu, got);
                const int off = g * (kBM * 128) + r * 128;
                const uint8_t *orow = o_s + off, *drow = smem + L::kDoOff + (n & 1) * L::kQBytes + off;
                if (ok) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const uint4 ov = *reinterpret_cast<const uint4 *>(orow + ((c ^ sw) << 4));
                        const uint4 dv = *reinterpret_cast<const uint4 *>(drow + ((c ^ sw) << 4));
                        const uint32_t ow[4] = {ov.x, ov.y, ov.z, ov.w}, dw[4] = {dv.x, dv.y, dv.z, dv.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 of = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&ow[e]));
                            const float2 df = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&dw[e]));
                            delta = fmaf(of.x, df.x, delta);
                            delta = fmaf(of.y, df.y, delta);
                        }
                    }
                }
            }
            delta_s[g * kBM + r] = delta;
            warp_arrive(qo_empty);  // this warp has read Q and O
            if (!(ok = all_ok(ok))) break;
            delta = delta_s[r] + delta_s[kBM + r];
            if (w.pos0 < kExactDelta) launch_dependent_wait();  // win_delta.cu's results
            if (valid && w.pos0 + r < kExactDelta)
                delta = a.delta[(size_t)w.bh * a.N + row];
            else if (valid && g == 0)
                a.delta[(size_t)w.bh * a.N + row] = delta;
            const uint64_t nl2 = f2_pack(-lse2, -lse2), d2 = f2_pack(delta, delta);
            for (int j = 0; j < w.span.n; ++j, ++t) {
                const uint32_t b = t & 1;
                ok = mbar_wait(&s_full[b], (t >> 1) & 1, a.status, kSiteSFull);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                tc_fence_after();
                const int key0 = w.span.key0(j, kBN) + g * kHalf;
                const int window = w.span.window_in(j, a.win.window);
                const bool need_mask = !all_seen(w.pos0 + quarter * 32, w.pos0 + quarter * 32 + 31, key0, key0 + kHalf - 1,
                                                  window, a.win.sinks);
                static_assert(kHalf == 32, "one mask word per thread and tile");
                const uint32_t seen = need_mask ? seen_keys(w.pos0 + r, key0, window, a.win.sinks) : 0u;
                // dS[b] was last read by the dQ product of step t-2
                if (t >= 2) {
                    ok = mbar_wait(&dq_done[b], ((t - 2) >> 1) & 1, a.status, kSiteDqDone);
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    tc_fence_after();
                }
                uint32_t sraw[kHalf], praw[kHalf], dsk[kHalf / 2];
                tmem_ld32(tmem + lane_base + 64 * b + g * kHalf, sraw);
                tmem_ld32(tmem + lane_base + kColDP + 64 * b + g * kHalf, praw);
                tmem_wait_ld();
                // dS / scale = P (dP - D), two scores per instruction
#pragma unroll
                for (int i = 0; i < kHalf; i += 2) {
                    float p0, p1;
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(sraw[i]), __uint_as_float(sraw[i + 1])), c2, nl2), p0, p1);
                    p0 = ex2_approx(p0);
                    p1 = ex2_approx(p1);
                    if (need_mask) {
                        if (!(seen & (1u << i))) p0 = 0.f;
                        if (!(seen & (2u << i))) p1 = 0.f;
                    }
                    dsk[i / 2] = f2_to_bf16x2(
                        f2_mul(f2_sub(f2_pack(__uint_as_float(praw[i]), __uint_as_float(praw[i + 1])), d2), f2_pack(p0, p1)));
                }
                tmem_st_n<kHalf / 2>(tmem + lane_base + kColDS + 32 * b + g * (kHalf / 2), dsk);
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(&ds_full[b]);
            }
            prev = w;
            ++n;
        }
        if (!dead && all_ok(ok) && n > 0) epilogue(n - 1, prev);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace

cudaError_t launch_win_dq(const BwdArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                          const CUtensorMap &tdo, const CUtensorMap &to, const CUtensorMap &tdq, int num_sms,
                          bool behind, cudaStream_t s) {
    if (kernel_head_dim(a.D) == 64) return launch_win_dq_k128(a, tq, tk, tv, tdo, to, tdq, num_sms, behind, s);
    if (kernel_head_dim(a.D) != kD) return launch_bwd_dq(a, tq, tk, tv, tdo, to, tdq, s, true, behind);
    static std::atomic<unsigned long long> allowed{0};
    cudaError_t e = allow_smem((const void *)win_dq_kernel, WinDqSmem::kAlloc, allowed);
    if (e != cudaSuccess) return e;
    const int n_items = (a.N + kBM - 1) / kBM * a.H * a.B;
    const int sms = num_sms > 0 ? num_sms : kNumSms;
    return launch_behind(win_dq_kernel, dim3(n_items < sms ? n_items : sms), kThreads, WinDqSmem::kAlloc, behind, 1, s, tq, tk,
                         tv, tdo, to, tdq, a, n_items);
}

}  // namespace fa
