// win_dq_k128.cu -- dQ of windowed attention for D = 64.  Per 128-row query tile, over
// the key tiles that its rows see (key_span):
//
//   D_i = sum_d dO_id O_id (written out),
//   S = Q K_j^T,  P = 2^(c S - L log2 e),  dP = dO V_j^T,  dS = P (dP - D),
//   dQ += dS K_j  (times scale at the end)
//
// Products, TMEM layout and compute warps are bwd_dq_k128.cu's: 128-key tiles, S and dP
// in one buffer each that the compute warps empty first thing, dS in two, Q and dO as
// TMEM operands; warp 0 TMA producer, warp 1 issuer A (S, dP), warp 2 issuer B (dQ),
// warps 3-18 compute, a thread owning one row and 32 keys of every tile; warp 19 stores
// (TMA).
//
// The walk is win_dq.cu's: one CTA per SM takes tiles in turn, the next one's Q, dO and
// O are loaded meanwhile, and once the compute warps have seen a tile's last dP they copy
// the next tile's Q and dO into TMEM and work on its first step before they read dQ.  They
// never meet at a barrier of all of them, and the producer works the tiles out for them.
// Sinks that fit into 32 columns are a product of 32 keys (idesc_sink), which only the
// first warpgroup works on.
// Bound by the chain S, dP -> compute -> dQ, a step of 128 keys in 0.9 us: B1 H32 N32768
// window 512, 1 sink: 346 us, 592 TFLOP/s of the visible pairs (three products each);
// B1 H8 N16384 window 2048: 113 us, 910.  bwd_dq.cu's 64-key tiles with two CTAs an SM
// took 347 and 121 (and 24.6 instead of 26 at window 128), a persistent grid of those 378.
#include "fa_internal.h"
#include "launch.cuh"
#include "sm100_ptx.cuh"
#include "win.cuh"
#include <cmath>

namespace fa {
namespace {

constexpr int kD = 64;
constexpr int kBM = 128;  // queries per item (TMEM lanes)
constexpr int kBN = 128;  // keys per tile
constexpr int kComputeWG = 4;
constexpr int kSpan = kBN / kComputeWG;  // 32 keys per compute thread and tile
constexpr int kFirstComputeWarp = 3;
constexpr int kComputeWarps = 4 * kComputeWG;
constexpr int kStoreWarp = kFirstComputeWarp + kComputeWarps;
constexpr int kThreads = 32 * (kStoreWarp + 1);
constexpr int kSlots = 8;  // K_j / V_j ring
constexpr int kSinkCols = 32;
static_assert(kSinkCols == kSpan, "the first warpgroup's keys");

enum : int { kSiteQ = 281, kSiteSlotEmpty, kSiteSlotFull, kSiteSFull, kSiteDsFull, kSiteDq, kSiteFinal, kSiteDrain,
             kSiteDqDone, kSiteQt, kSiteAcc, kSiteQEmpty, kSiteFree, kSiteDelta, kSiteStage };

struct K128Smem {
    static constexpr int kQBytes = kBM * kD * 2;
    static constexpr int kTileBytes = kBN * kD * 2;
    static constexpr int kQOff = 0, kDoOff = kQBytes, kOOff = 2 * kQBytes;
    static constexpr int kStageOff = 3 * kQBytes;  // dQ for its store (bf16: one panel, fp32: two)
    static constexpr int kSlotOff = 5 * kQBytes;
    static constexpr int kDeltaOff = kSlotOff + kSlots * kTileBytes;  // [2][kComputeWG][kBM] partial sums
    static constexpr int kItemOff = kDeltaOff + 2 * kComputeWG * kBM * 4;
    static constexpr int kBarOff = kItemOff + 32;
    // in_full, in_empty, slot_full/empty[kSlots], s_full, s_free, dp_full, dp_free, ds_full[2], dq_done[2], qt_ready,
    // acc_full, acc_free, final, a_final, delta_full, stage_full, stage_free
    static constexpr int kNumBars = 2 + 2 * kSlots + 16;
    static constexpr int kTmemHolderOff = kBarOff + kNumBars * 8;
    static constexpr int kAlloc = kTmemHolderOff + 16 + 1024;
    static_assert(kAlloc <= 232448, "shared memory budget");
};

__global__ void __launch_bounds__(kThreads, 1)
    win_dq_k128_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                  const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_do,
                  const __grid_constant__ CUtensorMap tmap_o, const __grid_constant__ CUtensorMap tmap_dq, BwdArgs a,
                  int n_items) {
    using L = K128Smem;
    constexpr uint32_t kTmemCols = 512;
    // S [0, 128), dP [128, 256), dS[b] [256 + 64b, +64), dQ [384, 448), Q [448, 480), dO [480, 512)
    constexpr uint32_t kColDP = 128, kColDS = 256, kColDQ = 384, kColQ = 448, kColDO = 480;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *q_s = smem + L::kQOff, *do_s = smem + L::kDoOff, *o_s = smem + L::kOOff;
    uint8_t *slots = smem + L::kSlotOff;
    float *delta_s = reinterpret_cast<float *>(smem + L::kDeltaOff);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBarOff);
    uint64_t *in_full = bars;                  // item n's Q, dO and O landed
    uint64_t *in_empty = in_full + 1;          // every compute warp has read them
    uint64_t *slot_full = in_empty + 1;
    uint64_t *slot_empty = slot_full + kSlots;
    uint64_t *s_full = slot_empty + kSlots;    // S of step t complete (steps counted across items)
    uint64_t *s_free = s_full + 1;             // every compute warp has loaded it
    uint64_t *dp_full = s_free + 1, *dp_free = dp_full + 1;
    uint64_t *ds_full = dp_free + 1;           // [2]: dS of step t written
    uint64_t *dq_done = ds_full + 2;           // [2]: dQ product of step t complete
    uint64_t *qt_ready = dq_done + 2;          // item n's Q and dO are in TMEM
    uint64_t *acc_full = qt_ready + 1;         // item n's dQ is complete
    uint64_t *acc_free = acc_full + 1;         // every compute warp has read it
    uint64_t *final_bar = acc_free + 1;
    uint64_t *a_final = final_bar + 1;
    uint64_t *delta_full = a_final + 1;        // item n's partial sums of D are in delta_s[n % 2]
    uint64_t *stage_full = delta_full + 1, *stage_free = stage_full + 1;  // item n's dQ is staged; its store has read it
    // what the compute warps need of item n: written before in_full's arrival, read before in_empty's
    int4 *item_s = reinterpret_cast<int4 *>(smem + L::kItemOff);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + L::kTmemHolderOff);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(in_full, 1);
        mbar_init(in_empty, kComputeWarps);
        mbar_init(s_full, 1);
        mbar_init(s_free, kComputeWarps);
        mbar_init(dp_full, 1);
        mbar_init(dp_free, kComputeWarps);
        for (int b = 0; b < 2; ++b) {
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
        mbar_init(delta_full, kComputeWarps);
        mbar_init(stage_full, kComputeWarps);
        mbar_init(stage_free, 1);
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
    // the sinks fit into 32 columns: sink tiles are products of 32 keys
    const bool few = a.win.sinks <= kSinkCols;

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
            int n = 0, t = 0;
            for (int k = 0; ok && k * (int)gridDim.x < n_items; ++k) {
                const int x = persistent_work_index(k, n_items);
                if (x < 0) continue;
                const WinRowItem w = win_row_item(a, x, kBM, kBN);
                if (n >= 1 && !(ok = mbar_wait(in_empty, (n - 1) & 1, a.status, kSiteQEmpty))) break;
                item_s[0] = make_int4(w.bh, w.row0, w.pos0, w.span.n);
                item_s[1] = make_int4(w.span.n_sink, w.span.lo, 0, 0);
                mbar_arrive_expect_tx(in_full, 3 * L::kQBytes);
                tma_load_3d(q_s, &tmap_q, in_full, 0, w.row0, w.bh);
                tma_load_3d(do_s, &tmap_do, in_full, 0, w.row0, w.bh);
                tma_load_3d(o_s, &tmap_o, in_full, 0, w.row0, w.bh);
                ++n;
                for (int j = 0; ok && j < w.span.n; ++j, ++t) {
                    const int key0 = w.span.key0(j, kBN);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // K_j, V_j
                        const int idx = 2 * t + h, slot = idx % kSlots, round = idx / kSlots;
                        if (!(ok = mbar_wait(&slot_empty[slot], (round & 1) ^ 1, a.status, kSiteSlotEmpty))) break;
                        mbar_arrive_expect_tx(&slot_full[slot], L::kTileBytes);
                        tma_load_3d(slots + slot * L::kTileBytes, h ? &tmap_v : &tmap_k, &slot_full[slot], 0, key0, w.kv_bh);
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
            if (n >= 1) mbar_wait(in_full, (n - 1) & 1, a.status, kSiteDrain);
        }
        __syncwarp();
    } else if (warp == 1) {
        // Issuer A: S = Q K_j^T and dP = dO V_j^T (Q and dO from TMEM), each into its one buffer as soon as every compute
        // warp has loaded the step before's.
        constexpr uint32_t idesc_sq = idesc_bf16_f32(kBM, kBN, false, false);
        constexpr uint32_t idesc_sink = idesc_bf16_f32(kBM, kSinkCols, false, false);
        const uint32_t slot_addr = smem_u32(slots);
        const bool leader = elect_one();
        bool ok = true;
        int n = 0, t = 0;
        for (int k = 0; ok && k * (int)gridDim.x < n_items; ++k) {
            const int x = persistent_work_index(k, n_items);
            if (x < 0) continue;
            const WinRowItem w = win_row_item(a, x, kBM, kBN);
            if (!(ok = warp_wait(qt_ready, n & 1, a.status, kSiteQt))) break;
            ++n;
            const bool sink_step = few && w.span.n_sink > 0;
            if (sink_step) {  // (apart from the loop, whose products' shape stays a constant: selecting it cost 4-6 % of all steps)
                const int k_slot = (2 * t) % kSlots, v_slot = (2 * t + 1) % kSlots;
                if (!(ok = warp_wait(&slot_full[k_slot], (2 * t / kSlots) & 1, a.status, kSiteSlotFull))) break;
                if (t >= 1 && !(ok = warp_wait(s_free, (t - 1) & 1, a.status, kSiteFree))) break;
                tc_fence_after();
                const uint64_t k_desc = sdesc_sw128(slot_addr + k_slot * L::kTileBytes, 16, 1024);
                if (leader) {
#pragma unroll
                    for (int ks = 0; ks < kD / 16; ++ks)
                        mma_ts(tmem, tmem + kColQ + ks * 8, sdesc_add(k_desc, ks * 32), idesc_sink, ks > 0);
                    mma_commit(s_full);
                }
                __syncwarp();
                if (!(ok = warp_wait(&slot_full[v_slot], ((2 * t + 1) / kSlots) & 1, a.status, kSiteSlotFull))) break;
                if (t >= 1 && !(ok = warp_wait(dp_free, (t - 1) & 1, a.status, kSiteFree))) break;
                tc_fence_after();
                const uint64_t v_desc = sdesc_sw128(slot_addr + v_slot * L::kTileBytes, 16, 1024);
                if (leader) {
#pragma unroll
                    for (int ks = 0; ks < kD / 16; ++ks)
                        mma_ts(tmem + kColDP, tmem + kColDO + ks * 8, sdesc_add(v_desc, ks * 32), idesc_sink, ks > 0);
                    mma_commit(dp_full);
                    mma_commit(&slot_empty[v_slot]);  // V_j is no longer needed
                }
                __syncwarp();
                ++t;
            }
            for (int j = sink_step ? 1 : 0; j < w.span.n; ++j, ++t) {
                const int k_slot = (2 * t) % kSlots, v_slot = (2 * t + 1) % kSlots;
                if (!(ok = warp_wait(&slot_full[k_slot], (2 * t / kSlots) & 1, a.status, kSiteSlotFull))) break;
                if (t >= 1 && !(ok = warp_wait(s_free, (t - 1) & 1, a.status, kSiteFree))) break;
                tc_fence_after();
                const uint64_t k_desc = sdesc_sw128(slot_addr + k_slot * L::kTileBytes, 16, 1024);
                if (leader) {
#pragma unroll
                    for (int ks = 0; ks < kD / 16; ++ks)
                        mma_ts(tmem, tmem + kColQ + ks * 8, sdesc_add(k_desc, ks * 32), idesc_sq, ks > 0);
                    mma_commit(s_full);
                }
                __syncwarp();
                if (!(ok = warp_wait(&slot_full[v_slot], ((2 * t + 1) / kSlots) & 1, a.status, kSiteSlotFull))) break;
                if (t >= 1 && !(ok = warp_wait(dp_free, (t - 1) & 1, a.status, kSiteFree))) break;
                tc_fence_after();
                const uint64_t v_desc = sdesc_sw128(slot_addr + v_slot * L::kTileBytes, 16, 1024);
                if (leader) {
#pragma unroll
                    for (int ks = 0; ks < kD / 16; ++ks)
                        mma_ts(tmem + kColDP, tmem + kColDO + ks * 8, sdesc_add(v_desc, ks * 32), idesc_sq, ks > 0);
                    mma_commit(dp_full);
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
            const bool sink_step = few && w.span.n_sink > 0;
            if (sink_step) {
                const uint32_t b = t & 1;
                const int k_slot = (2 * t) % kSlots;
                const uint64_t kmn_desc = sdesc_sw128(slot_addr + k_slot * L::kTileBytes, kBN * 128, 1024);
                if (!(ok = warp_wait(&ds_full[b], (t >> 1) & 1, a.status, kSiteDsFull))) break;
                // the first product overwrites dQ, which the item before's epilogue reads
                if (n >= 1 && !(ok = warp_wait(acc_free, (n - 1) & 1, a.status, kSiteAcc))) break;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < kSinkCols / 16; ++kk)
                        mma_ts(tmem + kColDQ, tmem + kColDS + 64 * b + kk * 8, sdesc_add(kmn_desc, kk * 2048), idesc_dq,
                               kk > 0);
                    mma_commit(&dq_done[b]);
                    mma_commit(&slot_empty[k_slot]);  // S completed before dS was written
                }
                __syncwarp();
                ++t;
            }
            for (int j = sink_step ? 1 : 0; j < w.span.n; ++j, ++t) {
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
                        mma_ts(tmem + kColDQ, tmem + kColDS + 64 * b + kk * 8, sdesc_add(kmn_desc, kk * 2048), idesc_dq,
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
    } else if (warp == kStoreWarp) {
        // Stores the dQ that the compute warps stage; TMA stores clip rows past N and columns past the caller's D.
        if (lane == 0) {
            int n = 0;
            const int pw = a.grad_bf16 ? 64 : 32;
            for (int k = 0; k * (int)gridDim.x < n_items; ++k) {
                const int x = persistent_work_index(k, n_items);
                if (x < 0) continue;
                const WinRowItem w = win_row_item(a, x, kBM, kBN);
                if (!mbar_wait(stage_full, n & 1, a.status, kSiteStage)) break;
                for (int col = 0; col < a.D; col += pw)
                    tma_store_3d(&tmap_dq, smem + L::kStageOff + col / pw * (kBM * 128), col, w.row0, w.bh);
                tma_store_commit();
                tma_store_wait_read();  // (and the CTA's shared memory must outlive the reads)
                mbar_arrive(stage_free);
                ++n;
            }
        }
        __syncwarp();
    } else {
        const int quarter = warp & 3;
        const int g = (warp - kFirstComputeWarp) >> 2;  // key range of every tile
        const int r = quarter * 32 + lane;
        const int sw = r & 7;
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        const uint64_t c2 = f2_pack(a.scale_log2, a.scale_log2);
        // Item n's dQ (times the scale), staged as 128-byte-swizzled panels of 128 rows (64 bf16 or 32 fp32 columns).
        auto epilogue = [&](int n) {
            bool good = mbar_wait(acc_full, n & 1, a.status, kSiteDq);
            if (!__all_sync(0xffffffffu, good)) return false;
            tc_fence_after();
            uint32_t v[16];
            tmem_ld16(tmem + lane_base + kColDQ + 16 * g, v);  // this warpgroup's columns
            tmem_wait_ld();
            tc_fence_before();
            warp_arrive(acc_free);
            if (n >= 1) good = mbar_wait(stage_free, (n - 1) & 1, a.status, kSiteStage);
            if (!__all_sync(0xffffffffu, good)) return false;
            uint8_t *stage = smem + L::kStageOff;
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * a.scale);
            if (a.grad_bf16) {
                uint8_t *prow = stage + r * 128;
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    st_shared_v4(prow + (((2 * g + c) ^ sw) << 4),
                                 pack_bf16x2(__uint_as_float(v[8 * c + 0]), __uint_as_float(v[8 * c + 1])),
                                 pack_bf16x2(__uint_as_float(v[8 * c + 2]), __uint_as_float(v[8 * c + 3])),
                                 pack_bf16x2(__uint_as_float(v[8 * c + 4]), __uint_as_float(v[8 * c + 5])),
                                 pack_bf16x2(__uint_as_float(v[8 * c + 6]), __uint_as_float(v[8 * c + 7])));
            } else {
                uint8_t *prow = stage + (g >> 1) * (kBM * 128) + r * 128;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    st_shared_v4(prow + (((4 * (g & 1) + c) ^ sw) << 4), v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
            }
            fence_proxy_async_smem();  // the staged panels are read by the TMA (async proxy)
            warp_arrive(stage_full);
            return true;
        };

        bool ok = true;
        int n = 0, t = 0;
        for (int k = 0; ok && k * (int)gridDim.x < n_items; ++k) {
            if (persistent_work_index(k, n_items) < 0) continue;
            ok = mbar_wait(in_full, n & 1, a.status, kSiteQ);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            const int4 i0 = item_s[0], i1 = item_s[1];
            const int pos0 = i0.z, row = i0.y + r;
            const KeySpan span{i1.x, i1.y, i0.w};
            const bool valid = row < a.N;
            const size_t at = (size_t)i0.x * a.N + (valid ? row : 0);
            // P = 2^(S c - L log2 e); rows past the last get P = 0
            const float lse = valid ? a.lse[at] : INFINITY;
            // Q (warpgroup 0) and dO (warpgroup 1) into TMEM as bf16 pairs (row r of the panel is 128 B at r * 128, its
            // 16-byte chunk c at c ^ (r % 8)); every S and dP product of the item before has completed
            if (g < 2) {
                const uint8_t *panel = (g == 0 ? q_s : do_s) + r * 128;
                uint32_t v[32];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(panel + ((c ^ sw) << 4));
                    v[4 * c] = u.x, v[4 * c + 1] = u.y, v[4 * c + 2] = u.z, v[4 * c + 3] = u.w;
                }
                tmem_st32(tmem + lane_base + (g == 0 ? kColQ : kColDO), v);
                tmem_wait_st();
            }
            tc_fence_before();
            warp_arrive(qt_ready);
            // D_i: warpgroup g sums columns [16g, 16g + 16); O's and dO's chunks sit at the same swizzled places.  (Every
            // warp had read the sums of item n - 2 when it added its own to those of item n - 1.)
            float *sums = delta_s + (n & 1) * (kComputeWG * kBM);
            float delta = 0.f;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int off = r * 128 + (((2 * g + c) ^ sw) << 4);
                const uint4 ov = *reinterpret_cast<const uint4 *>(o_s + off);
                const uint4 dv = *reinterpret_cast<const uint4 *>(do_s + off);
                const uint32_t ow[4] = {ov.x, ov.y, ov.z, ov.w}, dw[4] = {dv.x, dv.y, dv.z, dv.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 of = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&ow[e]));
                    const float2 df = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&dw[e]));
                    delta = fmaf(of.x, df.x, delta);
                    delta = fmaf(of.y, df.y, delta);
                }
            }
            sums[g * kBM + r] = delta;
            warp_arrive(in_empty);  // this warp has read Q, dO, O and the entry
            warp_arrive(delta_full);
            ok = mbar_wait(delta_full, n & 1, a.status, kSiteDelta);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            delta = 0.f;
#pragma unroll
            for (int u = 0; u < kComputeWG; ++u) delta += sums[u * kBM + r];
            if (pos0 < kExactDelta) launch_dependent_wait();  // win_delta.cu's results
            if (valid && pos0 + r < kExactDelta)
                delta = a.delta[at];
            else if (valid && g == 0)
                a.delta[at] = delta;
            const float lse2 = lse * 1.4426950408889634f;
            const uint64_t nl2 = f2_pack(-lse2, -lse2), d2 = f2_pack(delta, delta);
            int first = 0;
            if (few && span.n_sink > 0 && g > 0) {  // the step of 32 sinks is the first warpgroup's (a test in the loop: 3 %)
                const uint32_t b = t & 1;
                ok = mbar_wait(s_full, t & 1, a.status, kSiteSFull);
                warp_arrive(s_free);
                ok = ok && mbar_wait(dp_full, t & 1, a.status, kSiteSFull);
                warp_arrive(dp_free);
                if (t >= 2) ok = ok && mbar_wait(&dq_done[b], ((t - 2) >> 1) & 1, a.status, kSiteDqDone);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                warp_arrive(&ds_full[b]);
                if (n > 0 && !(ok = epilogue(n - 1))) break;
                first = 1;
                ++t;
            }
            for (int j = first; j < span.n; ++j, ++t) {
                const uint32_t b = t & 1;
                ok = mbar_wait(s_full, t & 1, a.status, kSiteSFull);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                tc_fence_after();
                uint32_t raw[kSpan], dsk[kSpan / 2];
                uint64_t p2[kSpan / 2];
                tmem_ld32(tmem + lane_base + g * kSpan, raw);
                tmem_wait_ld();
                tc_fence_before();
                warp_arrive(s_free);  // in registers: the next S may overwrite the buffer
                const int key0 = span.key0(j, kBN) + g * kSpan;
                const int window = span.window_in(j, a.win.window);
                const bool need_mask = !all_seen(pos0 + quarter * 32, pos0 + quarter * 32 + 31, key0, key0 + kSpan - 1,
                                                  window, a.win.sinks);
                // P while dP may still be executing, two scores per instruction
#pragma unroll
                for (int i = 0; i < kSpan; i += 2) {
                    float p0, p1;
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(raw[i]), __uint_as_float(raw[i + 1])), c2, nl2), p0, p1);
                    p2[i / 2] = f2_pack(ex2_approx(p0), ex2_approx(p1));
                }
                if (need_mask) {
                    const uint32_t seen = seen_keys(pos0 + r, key0, window, a.win.sinks);
#pragma unroll
                    for (int i = 0; i < kSpan; i += 2) {
                        float p0, p1;
                        f2_unpack(p2[i / 2], p0, p1);
                        if (!(seen & (1u << i))) p0 = 0.f;
                        if (!(seen & (2u << i))) p1 = 0.f;
                        p2[i / 2] = f2_pack(p0, p1);
                    }
                }
                ok = mbar_wait(dp_full, t & 1, a.status, kSiteSFull);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                tc_fence_after();
                tmem_ld32(tmem + lane_base + kColDP + g * kSpan, raw);
                tmem_wait_ld();
                tc_fence_before();
                warp_arrive(dp_free);
                // dS / scale = P (dP - D)
#pragma unroll
                for (int i = 0; i < kSpan; i += 2)
                    dsk[i / 2] = f2_to_bf16x2(
                        f2_mul(f2_sub(f2_pack(__uint_as_float(raw[i]), __uint_as_float(raw[i + 1])), d2), p2[i / 2]));
                // dS[b] was last read by the dQ product of step t-2
                if (t >= 2) {
                    ok = mbar_wait(&dq_done[b], ((t - 2) >> 1) & 1, a.status, kSiteDqDone);
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    tc_fence_after();
                }
                tmem_st16(tmem + lane_base + kColDS + 64 * b + 16 * g, dsk);
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(&ds_full[b]);
                if (j == 0 && n > 0 && !(ok = epilogue(n - 1))) break;
            }
            ++n;
        }
        if (ok && n > 0) epilogue(n - 1);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace

cudaError_t launch_win_dq_k128(const BwdArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                               const CUtensorMap &tdo, const CUtensorMap &to, const CUtensorMap &tdq, int num_sms,
                               bool behind, cudaStream_t s) {
    static std::atomic<unsigned long long> allowed{0};
    cudaError_t e = allow_smem((const void *)win_dq_k128_kernel, K128Smem::kAlloc, allowed);
    if (e != cudaSuccess) return e;
    const int n_items = (a.N + kBM - 1) / kBM * a.H * a.B;
    const int sms = num_sms > 0 ? num_sms : kNumSms;
    return launch_behind(win_dq_k128_kernel, dim3(n_items < sms ? n_items : sms), kThreads, K128Smem::kAlloc, behind, 1, s, tq,
                         tk, tv, tdo, to, tdq, a, n_items);
}

}  // namespace fa
