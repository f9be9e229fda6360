// win_dkdv.cu -- dK and dV of windowed attention for D = 64 and 128 (wider heads run
// bwd_dkdv.cu).  Per key tile of 128 keys, over the rows of every query head of
// its group whose window (or the sinks) holds one of the keys:
//
//   S^T = K Q_i^T,  P^T = 2^(c S^T - L_i log2 e),  dV += P^T dO_i,
//   dP^T = V dO_i^T,  dS^T = P^T (dP^T - D_i),     dK += dS^T Q_i  (times scale at the end)
//
// The products, the TMEM layouts and the roles are those of bwd_dkdv.cu (D = 128:
// 64-row query tiles, S^T and dP^T double-buffered) and bwd_dkdv_q128.cu (D = 64:
// 128-row tiles, S^T double-, dP^T single-buffered): warp 0 TMA producer and L / D
// ring, warp 1 issuer A (S^T, dP^T), warp 2 issuer B (dV, dK), warps 3-18 compute,
// a thread owning one key and a quarter of each tile's queries.
//
// What differs is the walk.  A window of 512 gives a key tile 5 query tiles, and a
// CTA's fixed cost (barriers, first loads, pipeline fill, epilogue: 7 us measured)
// was more than its 5 us of products.  So the grid is one CTA per SM that walks
// items: the producer loads the next item's K and V (two buffers) and query tiles,
// and issuer A runs its first products, while the compute warps still write the
// current item's gradients; only dV and dK in TMEM are handed over (acc_free).
// An item is a key tile, or a chunk of the rows behind a sink tile's window
// (win_key_item), whose fp32 partial sink_sum_kernel adds up; with few sinks those
// chunks can run in win_sinks.cu.  Bound by the compute
// warps (TMEM in, exponentials, TMEM out twice a tile) more than by the products:
// B2 H16/4 N4096 D128 window 1024: 146 us, 827 TFLOP/s of the visible pairs (four
// products each); B1 H32 N32768 D64 window 512: 405 us (and win_sinks.cu's 50 for one
// sink), 590 over both.
#include "fa_internal.h"
#include "launch.cuh"
#include "sm100_ptx.cuh"
#include "win.cuh"
#include <cmath>

namespace fa {
namespace {

constexpr int kBN = 128;  // keys per item (TMEM lanes)
constexpr int kComputeWG = 4;
constexpr int kFirstComputeWarp = 3;
constexpr int kComputeWarps = 4 * kComputeWG;
constexpr int kStoreWarp = kFirstComputeWarp + kComputeWarps;
constexpr int kThreads = 32 * (kStoreWarp + 1);

enum : int { kSiteKV = 221, kSiteSlotEmpty, kSiteSlotFull, kSiteSFull, kSitePReady, kSiteDpFull, kSiteDsReady, kSiteDone,
             kSiteFinal, kSiteDrain, kSiteStats, kSiteBuf, kSiteDpFree, kSiteAcc, kSiteKVEmpty, kSiteStage };

template <int D>
struct Dkdv {
    static constexpr int kBQ = D == 64 ? 128 : 64;        // queries per tile
    static constexpr int kSlots = D == 64 ? 9 : 6;        // Q_i / dO_i ring
    static constexpr int kStats = 2;                      // query tiles' L / D in flight: one beside each S^T buffer
    static constexpr int kSpan = kBQ / kComputeWG;        // queries per compute thread and tile
    static constexpr int kDpBufs = D == 64 ? 1 : 2;
    // TMEM columns: S^T[2], dP^T[kDpBufs] (kBQ each), dV, dK (D each).  P^T (bf16) goes over the first half of each
    // warpgroup's own S^T columns; dS^T over the second half (D = 64) or the first half of its dP^T columns.
    static constexpr uint32_t kColDP = 2 * kBQ, kColDV = kColDP + kDpBufs * kBQ, kColDK = kColDV + D;
    static constexpr uint32_t kColDS = kDpBufs == 1 ? kSpan / 2 : kColDP;  // + kBQ b + kSpan g
    static_assert(kColDK + D <= 512, "TMEM budget");
    static constexpr int kKVBytes = kBN * D * 2;
    static constexpr int kTileBytes = kBQ * D * 2;
    static constexpr int kSlotOff = 4 * kKVBytes;  // K, V of two items
    static constexpr int kStatOff = kSlotOff + kSlots * kTileBytes;  // [kStats][L kBQ | D kBQ] fp32
    static constexpr int kBarOff = kStatOff + kStats * 2 * kBQ * 4;
    // kv_full[2], kv_empty[2], slot_full/empty[kSlots], s_full[2], dp_full[2], p_ready[2], ds_ready[2], dv_done[2],
    // dk_done[2], dp_free, acc_full, acc_free, stage_full, stage_free, final, a_final
    static constexpr int kNumBars = 4 + 2 * kSlots + 12 + 7;
    static constexpr int kTmemHolderOff = kBarOff + kNumBars * 8;
    static constexpr int kAlloc = kTmemHolderOff + 16 + 1024;
    static_assert(kAlloc <= 232448, "shared memory budget");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    win_dkdv_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                    const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_do,
                    const __grid_constant__ CUtensorMap tmap_dk, const __grid_constant__ CUtensorMap tmap_dv,
                    const __grid_constant__ CUtensorMap tmap_pk, const __grid_constant__ CUtensorMap tmap_pv, BwdArgs a,
                    int n_items) {
    using C = Dkdv<D>;
    constexpr int kPanels = D / 64, kBQ = C::kBQ, NSLOT = C::kSlots, kSpan = C::kSpan;
    constexpr int kStepsPerWG = kSpan / 16;
    constexpr uint32_t kTmemCols = 512;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *slots = smem + C::kSlotOff;
    float *stat_s = reinterpret_cast<float *>(smem + C::kStatOff);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kBarOff);
    uint64_t *kv_full = bars;                   // [2]: item n's K, V landed in buffer n % 2
    uint64_t *kv_empty = kv_full + 2;           // [2]: item n's gradients, staged over K and V, have been stored
    uint64_t *slot_full = kv_empty + 2;
    uint64_t *slot_empty = slot_full + NSLOT;
    // [2]: S^T of step t is complete and the tile's L and D have landed (steps counted across items, b = t % 2)
    uint64_t *s_full = slot_empty + NSLOT;
    uint64_t *dp_full = s_full + 2;             // [kDpBufs]
    uint64_t *p_ready = dp_full + 2;            // [2]
    uint64_t *ds_ready = p_ready + 2;           // [2] (and every compute warp has read step t's L and D)
    uint64_t *dv_done = ds_ready + 2;           // [2]
    uint64_t *dk_done = dv_done + 2;            // [2]: and dV of that step (one issuer thread)
    uint64_t *dp_free = dk_done + 2;  // one dP^T buffer: every compute warp has loaded it
    uint64_t *acc_full = dp_free + 1;            // item n's dV and dK are complete
    uint64_t *acc_free = acc_full + 1;           // every compute warp has read them
    uint64_t *stage_full = acc_free + 1;         // every compute warp has staged its share of a gradient store
    uint64_t *stage_free = stage_full + 1;       // that store has read it
    uint64_t *final_bar = stage_free + 1;
    uint64_t *a_final = final_bar + 1;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + C::kTmemHolderOff);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int N = a.N;
    const int skip = D == 64 && a.win.few ? a.B * a.win.Hkv * a.win.chunks : 0;  // those run in win_sinks.cu
    if (threadIdx.x == 0) {
        for (int b = 0; b < 2; ++b) {
            mbar_init(&kv_full[b], 1);
            mbar_init(&kv_empty[b], 1);
            mbar_init(&s_full[b], 1 + 32);  // the commit, and one arrival per producer lane, when its copies have landed
            mbar_init(&dp_full[b], 1);
            mbar_init(&p_ready[b], kComputeWarps);  // one arrive per compute warp
            mbar_init(&ds_ready[b], kComputeWarps);
            mbar_init(&dv_done[b], 1);
            mbar_init(&dk_done[b], 1);
        }
        for (int s = 0; s < NSLOT; ++s) {
            mbar_init(&slot_full[s], 1);
            mbar_init(&slot_empty[s], 1);
        }
        mbar_init(dp_free, kComputeWarps);
        mbar_init(acc_full, 1);
        mbar_init(acc_free, kComputeWarps);
        mbar_init(stage_full, kComputeWarps);
        mbar_init(stage_free, 1);
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
    const uint32_t tmem = *tmem_holder;

    // Every role walks the same items: persistent_work_index deals them, n counts this CTA's.
    if (warp == 0) {
        if (lane == 0) {
            tma_prefetch_desc(&tmap_q);
            tma_prefetch_desc(&tmap_k);
            tma_prefetch_desc(&tmap_v);
            tma_prefetch_desc(&tmap_do);
        }
        int last_round[NSLOT];
#pragma unroll
        for (int s = 0; s < NSLOT; ++s) last_round[s] = -1;
        bool ok = true;
        int n = 0, t = 0;  // items, query tiles so far
        bool behind = true;
        for (int k = 0; ok && k * (int)gridDim.x < n_items; ++k) {
            const int x = persistent_work_index(k, n_items);
            if (x < 0) continue;
            const WinKeyItem w = win_key_item(a, x + skip, kBN, kBQ);
            const int buf = n & 1;
            if (n >= 2 && !(ok = warp_wait(&kv_empty[buf], ((n >> 1) - 1) & 1, a.status, kSiteKVEmpty))) break;
            if (lane == 0) {
                uint8_t *k_s = smem + buf * 2 * C::kKVBytes, *v_s = k_s + C::kKVBytes;
                mbar_arrive_expect_tx(&kv_full[buf], 2 * C::kKVBytes);
#pragma unroll
                for (int p = 0; p < kPanels; ++p) {
                    tma_load_3d(k_s + p * (kBN * 128), &tmap_k, &kv_full[buf], p * 64, w.k_tile * kBN, w.bh);
                    tma_load_3d(v_s + p * (kBN * 128), &tmap_v, &kv_full[buf], p * 64, w.k_tile * kBN, w.bh);
                }
            }
            ++n;
            WinRowWalk at(a, w);
            for (int i = 0; ok && i < w.n; ++i, ++t, at.next()) {
                const int q0 = w.rows.first + at.h * kBQ, slice = at.slice;
#pragma unroll
                for (int h = 0; h < 2; ++h) {  // Q_i, dO_i
                    const int idx = 2 * t + h, slot = idx % NSLOT, round = idx / NSLOT;
                    if (!(ok = warp_wait(&slot_empty[slot], (round & 1) ^ 1, a.status, kSiteSlotEmpty))) break;
                    if (lane == 0) {
                        uint8_t *dst = slots + slot * C::kTileBytes;
                        mbar_arrive_expect_tx(&slot_full[slot], C::kTileBytes);
#pragma unroll
                        for (int p = 0; p < kPanels; ++p)
                            tma_load_3d(dst + p * (kBQ * 128), h ? &tmap_do : &tmap_q, &slot_full[slot], p * 64, q0, slice);
                    }
#pragma unroll
                    for (int s = 0; s < NSLOT; ++s)
                        if (s == slot) last_round[s] = round;
                }
                if (!ok) break;
                // the tile's L_i and D_i: lane l copies words l, l + 32, ... of [L_i | D_i] (zeros past the last row)
                const int ss = t % C::kStats;
                if (t >= 2 && !(ok = warp_wait(&ds_ready[ss], ((t - 2) >> 1) & 1, a.status, kSiteStats))) break;
                // D comes from the dQ kernel, which may still run when this one was launched behind it.  The other
                // roles' bounded waits meanwhile span what is left of that kernel once it has SMs to spare: a query tile
                // or two of at most kMaxSum keys, 20 ms each.
                if (behind) launch_dependent_wait();
                behind = false;
                float *dst = stat_s + ss * 2 * kBQ;
#pragma unroll
                for (int e = 0; e < 2 * kBQ / 32; ++e) {
                    const int word = 32 * e + lane;
                    const bool is_l = e < kBQ / 32;
                    const int q = q0 + (is_l ? word : word - kBQ);
                    const bool valid = q < N;
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst + word)),
                                 "l"((is_l ? a.lse : a.delta) + (size_t)slice * N + (valid ? q : 0)), "r"(valid ? 4 : 0)
                                 : "memory");
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&s_full[ss]))
                             : "memory");
            }
        }
        // Drain: never leave the CTA with a copy still in flight.
        if (lane == 0) {
#pragma unroll
            for (int s = 0; s < NSLOT; ++s)
                if (last_round[s] >= 0) mbar_wait(&slot_full[s], last_round[s] & 1, a.status, kSiteDrain);
            if (n >= 2) mbar_wait(&kv_full[n & 1], ((n - 2) >> 1) & 1, a.status, kSiteDrain);
            if (n >= 1) mbar_wait(&kv_full[(n - 1) & 1], ((n - 1) >> 1) & 1, a.status, kSiteDrain);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
    } else if (warp == 1) {
        // Issuer A.  Each wait for a free buffer comes before the wait for the tile that goes into it.
        constexpr uint32_t idesc_s = idesc_bf16_f32(kBN, kBQ, false, false);  // S^T, dP^T
        const uint32_t slot_addr = smem_u32(slots);
        const bool leader = elect_one();
        bool ok = true;
        int n = 0, t = 0;
        for (int k = 0; ok && k * (int)gridDim.x < n_items; ++k) {
            const int x = persistent_work_index(k, n_items);
            if (x < 0) continue;
            const WinKeyItem w = win_key_item(a, x + skip, kBN, kBQ);
            const int buf = n & 1;
            if (!(ok = warp_wait(&kv_full[buf], (n >> 1) & 1, a.status, kSiteKV))) break;
            ++n;
            tc_fence_after();
            const uint32_t kv_addr = smem_u32(smem) + buf * 2 * C::kKVBytes;
            const uint64_t k_desc = sdesc_sw128(kv_addr, 16, 1024);
            const uint64_t v_desc = sdesc_sw128(kv_addr + C::kKVBytes, 16, 1024);
            for (int i = 0; i < w.n; ++i, ++t) {
                const int q_slot = (2 * t) % NSLOT, d_slot = (2 * t + 1) % NSLOT;
                const uint32_t b = t & 1, db = C::kDpBufs == 1 ? 0 : b;
                // S^T[b] last held step t-2's P^T (and, with one dP^T buffer, dS^T)
                if (t >= 2 && !(ok = warp_wait(C::kDpBufs == 1 ? &dk_done[b] : &dv_done[b], ((t - 2) >> 1) & 1, a.status,
                                               kSiteBuf)))
                    break;
                if (!(ok = warp_wait(&slot_full[q_slot], ((2 * t) / NSLOT) & 1, a.status, kSiteSlotFull))) break;
                tc_fence_after();
                const uint64_t q_desc = sdesc_sw128(slot_addr + q_slot * C::kTileBytes, 16, 1024);
                if (leader) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        mma_ss(tmem + kBQ * b, sdesc_add(k_desc, (ks >> 2) * (kBN * 128) + (ks & 3) * 32),
                               sdesc_add(q_desc, (ks >> 2) * (kBQ * 128) + (ks & 3) * 32), idesc_s, ks > 0);
                    mma_commit(&s_full[b]);
                }
                __syncwarp();
                if (C::kDpBufs == 1) {
                    if (t >= 1 && !(ok = warp_wait(dp_free, (t - 1) & 1, a.status, kSiteDpFree))) break;
                } else {  // dP^T[b] last held step t-2's dS^T
                    if (t >= 2 && !(ok = warp_wait(&dk_done[b], ((t - 2) >> 1) & 1, a.status, kSiteBuf))) break;
                }
                if (!(ok = warp_wait(&slot_full[d_slot], ((2 * t + 1) / NSLOT) & 1, a.status, kSiteSlotFull))) break;
                tc_fence_after();
                const uint64_t do_desc = sdesc_sw128(slot_addr + d_slot * C::kTileBytes, 16, 1024);
                if (leader) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        mma_ss(tmem + C::kColDP + kBQ * db, sdesc_add(v_desc, (ks >> 2) * (kBN * 128) + (ks & 3) * 32),
                               sdesc_add(do_desc, (ks >> 2) * (kBQ * 128) + (ks & 3) * 32), idesc_s, ks > 0);
                    mma_commit(&dp_full[db]);
                }
                __syncwarp();
            }
        }
        // Drain this warp's MMAs before TMEM can be released (immediate in the normal path).
        if (leader) mma_commit(a_final);
        __syncwarp();
        warp_wait(a_final, 0, a.status, kSiteFinal);
    } else if (warp == 2) {
        // Issuer B: dV += P^T dO_i and dK += dS^T Q_i (dO_i, Q_i as MN-major B operands: queries are the reduction).
        constexpr uint32_t idesc_g = idesc_bf16_f32(kBN, D, false, true);
        const uint32_t slot_addr = smem_u32(slots);
        const bool leader = elect_one();
        bool ok = true;
        int n = 0, t = 0;
        for (int k = 0; ok && k * (int)gridDim.x < n_items; ++k) {
            const int x = persistent_work_index(k, n_items);
            if (x < 0) continue;
            const WinKeyItem w = win_key_item(a, x + skip, kBN, kBQ);
            auto acc_ready = [&] { return n == 0 || warp_wait(acc_free, (n - 1) & 1, a.status, kSiteAcc); };
            // an item without rows waits too: every phase of acc_free has to be waited for
            if (w.n == 0 && !(ok = acc_ready())) break;
            for (int i = 0; i < w.n; ++i, ++t) {
                const uint32_t b = t & 1;
                const int q_slot = (2 * t) % NSLOT, d_slot = (2 * t + 1) % NSLOT;
                const uint64_t qmn_desc = sdesc_sw128(slot_addr + q_slot * C::kTileBytes, kBQ * 128, 1024);
                const uint64_t dmn_desc = sdesc_sw128(slot_addr + d_slot * C::kTileBytes, kBQ * 128, 1024);
                const uint32_t p_col = tmem + kBQ * b, ds_col = tmem + C::kColDS + kBQ * b;
                if (!(ok = warp_wait(&p_ready[b], (t >> 1) & 1, a.status, kSitePReady))) break;
                // p_ready only proves Q_i landed: wait for dO_i as well
                if (!(ok = warp_wait(&slot_full[d_slot], ((2 * t + 1) / NSLOT) & 1, a.status, kSiteSlotFull))) break;
                // the item's first product overwrites dV (its later ones dK) that the item before's epilogue reads
                if (i == 0 && !(ok = acc_ready())) break;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < kBQ / 16; ++kk)
                        mma_ts(tmem + C::kColDV, p_col + (kk / kStepsPerWG) * kSpan + (kk % kStepsPerWG) * 8,
                               sdesc_add(dmn_desc, kk * 2048), idesc_g, (i > 0 || kk > 0));
                    mma_commit(&dv_done[b]);
                }
                __syncwarp();
                if (!(ok = warp_wait(&ds_ready[b], (t >> 1) & 1, a.status, kSiteDsReady))) break;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < kBQ / 16; ++kk)
                        mma_ts(tmem + C::kColDK, ds_col + (kk / kStepsPerWG) * kSpan + (kk % kStepsPerWG) * 8,
                               sdesc_add(qmn_desc, kk * 2048), idesc_g, (i > 0 || kk > 0));
                    mma_commit(&dk_done[b]);
                    // S^T_i and dP^T_i completed before dS^T_i was written: nothing reads Q_i or dO_i any more
                    mma_commit(&slot_empty[q_slot]);
                    mma_commit(&slot_empty[d_slot]);
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
        // Stores the gradients that the compute warps stage over an item's K and V, then hands that memory back.
        if (lane == 0) {
            bool ok = true;
            int n = 0, stores = 0;
            for (int k = 0; ok && k * (int)gridDim.x < n_items; ++k) {
                const int x = persistent_work_index(k, n_items);
                if (x < 0) continue;
                const WinKeyItem w = win_key_item(a, x + skip, kBN, kBQ);
                const bool partial = w.part >= 0, out_bf16 = a.grad_bf16 && !partial;
                const uint8_t *stage = smem + (n & 1) * 2 * C::kKVBytes;
                const int y = partial ? 0 : w.k_tile * kBN, z = partial ? w.part : w.bh;
                const int pw = out_bf16 ? 64 : 32, panels = D / pw;
                for (int which = out_bf16 ? 1 : 0; which < 2; ++which, ++stores) {
                    if (!(ok = mbar_wait(stage_full, stores & 1, a.status, kSiteStage))) break;
                    const CUtensorMap *m = which ? (partial ? &tmap_pk : &tmap_dk) : (partial ? &tmap_pv : &tmap_dv);
                    for (int p = 0; p < panels && p * pw < a.D; ++p) {
                        if (out_bf16) tma_store_3d(&tmap_dv, stage + p * (kBN * 128), p * pw, y, z);
                        tma_store_3d(m, stage + (out_bf16 ? C::kKVBytes : 0) + p * (kBN * 128), p * pw, y, z);
                    }
                    tma_store_commit();
                    tma_store_wait_read();  // (and the CTA's shared memory must outlive the reads)
                    mbar_arrive(stage_free);
                }
                if (ok) mbar_arrive(&kv_empty[n & 1]);
                ++n;
            }
        }
        __syncwarp();
    } else {
        const int quarter = warp & 3;
        const int g = (warp - kFirstComputeWarp) >> 2;  // query range of every tile
        const int r = quarter * 32 + lane;              // key row within the tile (TMEM lane)
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        constexpr float kLog2e = 1.4426950408889634f;
        const uint64_t c2 = f2_pack(a.scale_log2, a.scale_log2), nlog2e2 = f2_pack(-kLog2e, -kLog2e);
        bool ok = true;
        int n = 0, t = 0, stores = 0;
        const int off = a.win.Nk - N;
        // the next item is worked out while the current one's last products run
        int k = 0;
        auto next_item = [&](WinKeyItem *w) {
            for (; k * (int)gridDim.x < n_items; ++k) {
                const int x = persistent_work_index(k, n_items);
                if (x < 0) continue;
                *w = win_key_item(a, x + skip, kBN, kBQ);
                ++k;
                return true;
            }
            return false;
        };
        WinKeyItem w;
        bool more = next_item(&w);
        while (ok && more) {
            // the rows that see this thread's key: [lo, hi)
            const int key = w.k_tile * kBN + r;
            const int lo = key - off;
            const int hi = key >= a.win.Nk ? 0 : key < a.win.sinks ? N : min(N, key - off + a.win.window);
            WinRowWalk at(a, w);
            for (int i = 0; i < w.n; ++i, ++t, at.next()) {
                const uint32_t b = t & 1, db = C::kDpBufs == 1 ? 0 : b;
                const float4 *ls4 = reinterpret_cast<const float4 *>(stat_s + b * 2 * kBQ + g * kSpan);
                const float4 *ds4 = reinterpret_cast<const float4 *>(stat_s + b * 2 * kBQ + kBQ + g * kSpan);
                const int q0 = w.rows.first + at.h * kBQ + g * kSpan;  // first query of this thread's range
                const bool any_mask = __any_sync(0xffffffffu, q0 < lo || q0 + kSpan > hi);
                // None of this warp's keys is seen by any of its queries (along the edges of the band, and in the chunks behind
                // a sink tile): P^T and dS^T are zeros.  Step of 4096 rows, window 1024, D = 128: 157 -> 146 us; no
                // difference at D = 64, which has no registers left for it.
                const bool none = D == 128 && any_mask && __all_sync(0xffffffffu, q0 >= hi || q0 + kSpan <= lo);

                ok = mbar_wait(&s_full[b], (t >> 1) & 1, a.status, kSiteSFull);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                tc_fence_after();
                // P^T of this thread's queries: bf16 pairs for the dV product, fp32 pairs for dS^T (rounding both
                // factors would make dK's error a quarter larger)
                uint32_t pk[kSpan / 2];
                uint64_t p2[kSpan / 2];
                if (none) {
#pragma unroll
                    for (int e = 0; e < kSpan / 2; ++e) pk[e] = 0u;
                } else {
                    uint32_t raw[kSpan];
                    tmem_ld_n<kSpan>(tmem + lane_base + kBQ * b + g * kSpan, raw);
                    tmem_wait_ld();
#pragma unroll
                    for (int q4 = 0; q4 < kSpan / 4; ++q4) {
                        const float4 l4 = ls4[q4];  // natural-log L of four queries
                        float p[4];
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(raw[4 * q4 + 0]), __uint_as_float(raw[4 * q4 + 1])), c2,
                                         f2_mul(f2_pack(l4.x, l4.y), nlog2e2)),
                                  p[0], p[1]);
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(raw[4 * q4 + 2]), __uint_as_float(raw[4 * q4 + 3])), c2,
                                         f2_mul(f2_pack(l4.z, l4.w), nlog2e2)),
                                  p[2], p[3]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) p[e] = ex2_approx(p[e]);
                        p2[2 * q4] = f2_pack(p[0], p[1]);
                        p2[2 * q4 + 1] = f2_pack(p[2], p[3]);
                        pk[2 * q4] = pack_bf16x2(p[0], p[1]);
                        pk[2 * q4 + 1] = pack_bf16x2(p[2], p[3]);
                    }
                    if (any_mask) {
                        const uint32_t seen = ~low_bits(lo - q0) & low_bits(hi - q0);
#pragma unroll
                        for (int e = 0; e < kSpan / 2; ++e) {
                            float p0, p1;
                            f2_unpack(p2[e], p0, p1);
                            if (!(seen & (1u << (2 * e)))) p0 = 0.f;
                            if (!(seen & (2u << (2 * e)))) p1 = 0.f;
                            p2[e] = f2_pack(p0, p1);
                            pk[e] = pack_bf16x2(p0, p1);
                        }
                    }
                }
                tmem_st_n<kSpan / 2>(tmem + lane_base + kBQ * b + g * kSpan, pk);
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(&p_ready[b]);

                ok = mbar_wait(&dp_full[db], (C::kDpBufs == 1 ? t : t >> 1) & 1, a.status, kSiteDpFull);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                tc_fence_after();
                if (none) {
                    if constexpr (C::kDpBufs == 1) warp_arrive(dp_free);
                    tmem_st_n<kSpan / 2>(tmem + lane_base + C::kColDS + kBQ * b + g * kSpan, pk);
                } else {
                    uint32_t raw[kSpan], dsk[kSpan / 2];
                    tmem_ld_n<kSpan>(tmem + lane_base + C::kColDP + kBQ * db + g * kSpan, raw);
                    tmem_wait_ld();
                    if constexpr (C::kDpBufs == 1) {  // in registers: the next dP^T may overwrite the buffer
                        tc_fence_before();
                        warp_arrive(dp_free);
                    }
#pragma unroll
                    for (int q4 = 0; q4 < kSpan / 4; ++q4) {
                        const float4 d4 = ds4[q4];
                        dsk[2 * q4] = f2_to_bf16x2(f2_mul(
                            f2_sub(f2_pack(__uint_as_float(raw[4 * q4 + 0]), __uint_as_float(raw[4 * q4 + 1])),
                                   f2_pack(d4.x, d4.y)),
                            p2[2 * q4]));
                        dsk[2 * q4 + 1] = f2_to_bf16x2(f2_mul(
                            f2_sub(f2_pack(__uint_as_float(raw[4 * q4 + 2]), __uint_as_float(raw[4 * q4 + 3])),
                                   f2_pack(d4.z, d4.w)),
                            p2[2 * q4 + 1]));
                    }
                    tmem_st_n<kSpan / 2>(tmem + lane_base + C::kColDS + kBQ * b + g * kSpan, dsk);
                }
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(&ds_ready[b]);
            }
            WinKeyItem nw;
            more = next_item(&nw);
            if (ok) ok = mbar_wait(acc_full, n & 1, a.status, kSiteDone);
            // K and V have landed (with no query tile nothing has waited for them): their memory is the staging area
            if (ok) ok = mbar_wait(&kv_full[n & 1], (n >> 1) & 1, a.status, kSiteKV);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            tc_fence_after();
            // Epilogue: dV, then dK (times the scale its dS^T left out) as 128-byte-swizzled panels of 128 rows (64
            // bf16 or 32 fp32 columns) over this item's K and V, for the store warp's TMA stores, which clip rows past Nk
            // and columns past the caller's D.  bf16: both in one store; fp32 fills the area twice.
            const bool out_bf16 = a.grad_bf16 && w.part < 0;
            uint8_t *stage = smem + (n & 1) * 2 * C::kKVBytes;
            constexpr int kCols = D / kComputeWG;  // this warpgroup's columns of each gradient (16 or 32)
            const int c0 = g * kCols, sw = r & 7;
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                uint8_t *area = stage + (out_bf16 ? which * C::kKVBytes : 0) + r * 128;
                uint32_t v[kCols];
                tmem_ld_n<kCols>(tmem + lane_base + (which ? C::kColDK : C::kColDV) + c0, v);
                tmem_wait_ld();
                if (which == 1) {
                    tc_fence_before();
                    warp_arrive(acc_free);
                }
                // The store before has read its area (of this item's: the same one).  Every store's phase is waited
                // for: a phase passed over would let a later wait through one store early.
                if ((which == 0 || !out_bf16) && stores >= 1) {
                    ok = mbar_wait(stage_free, (stores - 1) & 1, a.status, kSiteStage);
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                }
                const float osc = which ? a.scale : 1.f;
#pragma unroll
                for (int e = 0; e < kCols; ++e) v[e] = w.n == 0 ? 0u : __float_as_uint(__uint_as_float(v[e]) * osc);
                if (out_bf16) {
                    uint8_t *prow = area + (c0 / 64) * (kBN * 128);
                    const int cb = (c0 % 64) / 8;
#pragma unroll
                    for (int c = 0; c < kCols / 8; ++c)
                        st_shared_v4(prow + (((cb + c) ^ sw) << 4),
                                     pack_bf16x2(__uint_as_float(v[8 * c + 0]), __uint_as_float(v[8 * c + 1])),
                                     pack_bf16x2(__uint_as_float(v[8 * c + 2]), __uint_as_float(v[8 * c + 3])),
                                     pack_bf16x2(__uint_as_float(v[8 * c + 4]), __uint_as_float(v[8 * c + 5])),
                                     pack_bf16x2(__uint_as_float(v[8 * c + 6]), __uint_as_float(v[8 * c + 7])));
                } else {
                    uint8_t *prow = area + (c0 / 32) * (kBN * 128);
                    const int cb = (c0 % 32) / 4;
#pragma unroll
                    for (int c = 0; c < kCols / 4; ++c)
                        st_shared_v4(prow + (((cb + c) ^ sw) << 4), v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
                }
                if (which == 1 || !out_bf16) {
                    fence_proxy_async_smem();  // the staged tile is read by the TMA (async proxy)
                    warp_arrive(stage_full);
                    ++stores;
                }
            }
            w = nw;
            ++n;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Adds the partials of one sink tile (its own rows', then the chunks', in that order) into dK and dV; four columns a
// thread.  partials of a tile: [part][128][D].
__global__ void sink_sum_kernel(BwdArgs a, const float *part_dk, const float *part_dv) {
    launch_dependent_wait();
    const int cols = a.D / 4, parts = 1 + a.win.chunks;
    const int tile = blockIdx.y;  // (key slice, sink tile)
    const int bh = tile / a.win.sink_tiles, k0 = tile % a.win.sink_tiles * kBN;
    const int rows = min(kBN, a.win.Nk - k0);
    for (int e = blockIdx.x * blockDim.x + threadIdx.x; e < rows * cols; e += gridDim.x * blockDim.x) {
        const size_t in = (size_t)tile * parts * kBN * a.D + (size_t)e * 4;
        const size_t out = ((size_t)bh * a.win.Nk + k0) * a.D + (size_t)e * 4;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const float *src = (w ? part_dv : part_dk) + in;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            const int n = a.win.few && e / cols >= kFewSinks ? 1 : parts;  // the others of win_sinks.cu hold 16 rows
#pragma unroll 4
            for (int p = 0; p < n; ++p) {
                const float4 v = *reinterpret_cast<const float4 *>(src + (size_t)p * kBN * a.D);
                s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
            }
            void *dst = w ? a.dv : a.dk;
            if (a.grad_bf16)
                *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(dst) + out) =
                    make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
            else
                *reinterpret_cast<float4 *>(static_cast<float *>(dst) + out) = s;
        }
    }
}

template <int D>
cudaError_t launch_items(const BwdArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                         const CUtensorMap &tdo, const CUtensorMap &tdk, const CUtensorMap &tdv, const CUtensorMap *parts,
                         int num_sms, bool behind, cudaStream_t s) {
    using C = Dkdv<D>;
    auto kern = win_dkdv_kernel<D>;
    static std::atomic<unsigned long long> allowed{0};
    cudaError_t e = allow_smem((const void *)kern, C::kAlloc, allowed);
    if (e != cudaSuccess) return e;
    const int chunks = a.win.few ? 0 : a.win.sink_tiles * a.win.chunks;
    const int n_items = ((a.win.Nk + kBN - 1) / kBN + chunks) * a.win.Hkv * a.B;
    const int sms = num_sms > 0 ? num_sms : kNumSms;
    return launch_behind(kern, dim3(n_items < sms ? n_items : sms), kThreads, C::kAlloc, behind, 1, s, tq, tk, tv, tdo, tdk,
                         tdv, parts[0], parts[1], a, n_items);
}

}  // namespace

cudaError_t launch_sink_sum(const BwdArgs &a, const float *part_dk, const float *part_dv, cudaStream_t s) {
    const dim3 grid((kBN * a.D / 4 + 255) / 256, a.B * a.win.Hkv * a.win.sink_tiles);
    return launch_behind(sink_sum_kernel, grid, 256, 0, true, 1, s, a, part_dk, part_dv);
}

cudaError_t launch_win_dkdv(const BwdArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                            const CUtensorMap &tdo, const CUtensorMap &tdk, const CUtensorMap &tdv,
                            const CUtensorMap *parts, int num_sms, bool behind, cudaStream_t s) {
    switch (kernel_head_dim(a.D)) {
        case 64: return launch_items<64>(a, tq, tk, tv, tdo, tdk, tdv, parts, num_sms, behind, s);
        case 128: return launch_items<128>(a, tq, tk, tv, tdo, tdk, tdv, parts, num_sms, behind, s);
        default: return launch_bwd_dkdv(a, tq, tk, tv, tdo, tdk, tdv, s, parts);
    }
}

}  // namespace fa
