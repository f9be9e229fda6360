// win_fwd.cu -- the forward over the keys that a span of query rows sees: windowed
// attention (window, sinks, grouped heads, a chunk of rows behind cached keys)
// and the shared prefix of a decode batch.  D = 64 and 128; wider heads run
// fwd_bf16.cu.
//
// Per row i at position p:  O = sum_j P_ij v_j / l,  P_ij = 2^(c s_ij - m) over the
// visible keys j <= p with j < sinks or j > p - window, m the running maximum
// (base 2, c = scale log2 e), l the running sum, L = (m + log2 l) ln 2.
//
// One tcgen05 issuer, one softmax warpgroup per 128-row query tile (a thread per row, its TMEM lane), a persistent grid
// past a TMA ring of K/V tiles.  Two forms:
//   window      one query tile a CTA and two CTAs an SM: while one waits at the end of a block or for a product, the
//               other's softmax has the SM.  S(j + 1) is issued before PV(j), P has columns of its own, the producer
//               works the blocks out ahead.  A block reads its sink tiles, then its window from the first key that its
//               first row sees (key_span); only tiles that hold a masked pair build masks.  (Two tiles past one stream of
//               keys, as the prefix form has them: 1197 us instead of 1035 for a 32K prompt at D = 64.)  Bound by the
//               chain S -> softmax -> PV: a tile's exponentials and conversions take ~1300 cycles with one warp a
//               scheduler (~1100 a tile with the other CTA's between them), and they begin when the PV before has
//               ended (p_free: there is one P), so the two overlap between the CTAs only.  No pipe is full (window 512,
//               D = 64: issue slots 50 %, XU 31 %, tensor 30 %; window 1024, D = 128: 41, 26, 46).  B1 H32/8 N32768 D64
//               window 4096: 1035 us, 997 TFLOP/s; B2 H16/4 N4096 D128 window 1024: 66 us, 920; B1 H32 N32768
//               D64 window 512: 253 us, 540.
//   prefix      128-row tiles packed from the rows of many sequences (the group's heads and the new rows of one
//               sequence are adjacent in memory, so one 4-D TMA box gathers them), two of them past one stream of
//               128-key tiles (one chunk of the prefix), P over S in TMEM; partials instead of O.  Bound by its products
//               and the softmax: 512 rows and 8 key heads against 32768 keys at D = 128, 1.7 us for a
//               chunk's key tile of two query tiles, 1500 TFLOP/s while it runs.
#include "fa_internal.h"
#include "launch.cuh"
#include "sm100_ptx.cuh"
#include "win.cuh"
#include <cmath>

namespace fa {
namespace {

constexpr int kBM = 128;            // rows per query tile (TMEM lanes)
constexpr int kFirstSoftmaxWarp = 2;

enum : int { kSiteQ = 181, kSiteSlotEmpty, kSiteSlotFull, kSiteSFull, kSitePFull, kSitePV, kSiteFinal, kSiteDrain,
             kSiteQEmpty, kSiteOFree, kSiteStage, kSiteBlock, kSiteSFree };

constexpr int kBlocks = 4;  // blocks that the producer has worked out ahead of the softmax warps

template <int D, int NSLOT, int kTiles, int kBN>
struct SpanSmem {
    static constexpr int kPanels = D / 64;
    static constexpr int kQBytes = kBM * D * 2;    // one query tile
    static constexpr int kSlotBytes = kBN * D * 2;  // one K or V tile
    // one tile a CTA (windowed): the next block's Q has a buffer of its own (D = 64), O is staged 64 columns at a time
    static constexpr int kQBufs = kTiles == 1 && D == 64 ? 2 : 1;
    static constexpr int kStageCols = kTiles == 1 ? 64 : 0;
    static constexpr int kThreads = 32 * kFirstSoftmaxWarp + 128 * kTiles;
    static constexpr int kQOff = 0;
    static constexpr int kSlotOff = kQBufs * kTiles * kQBytes;
    static constexpr int kStageOff = kSlotOff + NSLOT * kSlotBytes;  // 64 columns of O, staged for TMA stores
    static constexpr int kBarOff = kStageOff + kBM * kStageCols * 2;
    // q_full[2], q_empty[2], slot_full[NSLOT], slot_empty[NSLOT], per tile: s_full, p_full, pv_done, o_free; final,
    // stage_full, stage_free, s_free; block_full[kBlocks], block_empty[kBlocks]
    static constexpr int kNumBars = 4 + 2 * NSLOT + 4 * kTiles + 4 + 2 * kBlocks;
    static constexpr int kTmemHolderOff = kBarOff + kNumBars * 8;
    static constexpr int kBlockOff = (kTmemHolderOff + 16 + 15) / 16 * 16;  // SoftBlock [kBlocks][kTiles], 16-byte aligned
    static_assert(kBlockOff % 16 == 0 && kBarOff % 16 == 0, "vector accesses");
    static constexpr int kAlloc = kBlockOff + kBlocks * kTiles * 32;  // from a 1024-byte boundary
};

// The work of one block of this CTA: its query tiles and the key tiles that they read.  The producer and the issuer
// walk the same sequence of blocks and compute these alike.
template <int kTiles>
struct SpanBlock {
    KeySpan span;                // the key tiles
    int kv_bh, y_off;            // their K/V slice, and the row that key 0 of the span sits at
    int n[kTiles];               // key tiles that query tile x reads: span.n, or 0 where there is no such query tile
    int zq[kTiles], yq[kTiles];  // windowed: the tile's head slice and first row; prefix: chunk, packed tile
    int p0[kTiles];              // windowed: position of the tile's first row

    __device__ __forceinline__ bool reads(int x, int j) const { return j < n[x]; }
};

// Windowed blocks in longest-first order: the last rows of every head first.
template <int kBN>
__device__ __forceinline__ SpanBlock<1> window_block(const SpanArgs &a, int L) {
    SpanBlock<1> w;
    const int rank = a.per_rows.div(L), bh = L - rank * (int)a.per_rows.d;
    const int row0 = ((a.Nq + kBM - 1) / kBM - 1 - rank) * kBM;
    const int b = a.per_seq.div(bh), h = bh - b * (int)a.per_seq.d;
    const int off = a.Nk - a.Nq;
    w.kv_bh = b * a.Hkv + a.group.div(h);
    w.y_off = 0;
    w.zq[0] = bh;
    w.yq[0] = row0;
    w.p0[0] = off + row0;
    w.span = key_span(off + row0, off + min(a.Nq, row0 + kBM) - 1, a.window, a.sinks, kBN);
    w.n[0] = w.span.n;
    return w;
}

// Shared-prefix blocks: packed query tiles of a key head against one chunk of the prefix.
template <int kTiles, int kBN>
__device__ __forceinline__ SpanBlock<kTiles> prefix_block(const SpanArgs &a, int L) {
    SpanBlock<kTiles> w;
    const int groups = (a.parts.m_tiles + kTiles - 1) / kTiles;
    const int m = (L % groups) * kTiles;
    const int rest = L / groups;
    const int chunk = rest % a.parts.splits;
    w.kv_bh = rest / a.parts.splits;
    w.y_off = chunk * a.chunk_tiles * kBN;
    w.span.n_sink = 0;
    w.span.lo = 0;
    w.span.n = min(a.chunk_tiles, (a.Nk + kBN - 1) / kBN - chunk * a.chunk_tiles);
#pragma unroll
    for (int x = 0; x < kTiles; ++x) {
        w.zq[x] = chunk;
        w.yq[x] = m + x;
        w.p0[x] = 0;
        w.n[x] = m + x < a.parts.m_tiles ? w.span.n : 0;
    }
    return w;
}

template <bool PREFIX, int kTiles, int kBN>
__device__ __forceinline__ SpanBlock<kTiles> span_block(const SpanArgs &a, int L) {
    if constexpr (PREFIX) return prefix_block<kTiles, kBN>(a, L);
    else return window_block<kBN>(a, L);
}

// Columns of key tile j that are computed: all of them, or 32 of a sink tile whose sinks fit there.
template <bool PREFIX, int kBN>
__device__ __forceinline__ int tile_cols(const SpanArgs &a, int n_sink, int j) {
    return PREFIX || j >= n_sink || a.sinks - j * kBN > 32 ? kBN : 32;
}

// What the softmax of one query tile needs of a block.  The producer thread writes it, some blocks ahead: working it
// out (a handful of divisions and ranges) took each softmax warp 1000 cycles between two blocks.
struct __align__(16) SoftBlock {
    int n;             // key tiles that the query tile reads (-1: no more blocks)
    int n_sink, key0;  // the first n_sink are sink tiles; the next starts at key key0
    int use;           // windowed: blocks of this CTA before this one, each with an epilogue through the staging buffer
    int zq, yq, p0, kv_bh;
};
static_assert(sizeof(SoftBlock) == 32, "two 16-byte loads");

// First sequence and first row (of the R rows of a sequence and key head) of packed query tile t.
__device__ __forceinline__ void packed_tile(const SpanArgs &a, int t, int *b0, int *r0) {
    const int row_tiles = (a.parts.R + a.parts.rb - 1) / a.parts.rb;  // 1 unless a sequence alone has more than kBM rows
    *b0 = t / row_tiles * a.parts.nb;
    *r0 = t % row_tiles * a.parts.rb;
}

template <int kTiles>
__host__ __device__ inline int span_blocks(const SpanArgs &a, bool prefix) {
    if (prefix) return (a.parts.m_tiles + kTiles - 1) / kTiles * a.parts.splits * a.Hkv;
    return (a.Nq + kBM - 1) / kBM * (int)a.per_rows.d;
}

// Persistent: the grid has at most kCtas CTAs per SM, each walking its blocks in turn, so the next block's
// Q load and first S products overlap the previous block's last products and epilogue.  The K/V ring
// and every barrier's phase run on across blocks.
// kBN: keys per K/V tile.
template <int D, int NSLOT, bool PREFIX, int kTiles, int kCtas, int kBN>
__global__ void __launch_bounds__(32 * kFirstSoftmaxWarp + 128 * kTiles, kCtas)
    win_fwd_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                   const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_ks,
                   const __grid_constant__ CUtensorMap tmap_vs, const __grid_constant__ CUtensorMap tmap_o, SpanArgs a) {
    using L = SpanSmem<D, NSLOT, kTiles, kBN>;
    constexpr int kPanels = L::kPanels;
    constexpr uint32_t kTmemCols = 512 / kCtas;
    constexpr int kQBufs = L::kQBufs;
    // TMEM columns: S_A, S_B (P_X over the first kBN/2 columns of S_X), then O_A, O_B.  One tile a CTA: P has columns of its
    // own behind O, so that the next S runs while the softmax works on this one.
    constexpr bool kOwnP = kTiles == 1;
    constexpr uint32_t kColS = 0, kColO = kTiles * kBN, kColP = kOwnP ? kColO + D : kColS;
    static_assert(kColO + kTiles * D + (kOwnP ? kBN / 2 : 0) <= kTmemCols, "TMEM budget");

    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {  // the swizzled tiles need it, and there is no room to round up where two CTAs share an SM
        if (threadIdx.x == 0) record_failure(a.status, 5 /* FA_ERR_ALIGN */, kSiteQ);
        return;
    }
    uint8_t *q_s = smem + L::kQOff;
    uint8_t *slots = smem + L::kSlotOff;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::kBarOff);
    uint64_t *q_full = bars;                // [kQBufs]: block b's Q tiles landed (buffer b % kQBufs)
    uint64_t *q_empty = bars + 2;           // [kQBufs]: every S MMA of block b has completed
    uint64_t *slot_full = bars + 4;
    uint64_t *slot_empty = slot_full + NSLOT;
    uint64_t *s_full = slot_empty + NSLOT;  // [tile]: S_X of step g complete (phase g, steps counted across blocks)
    uint64_t *p_full = s_full + kTiles;     // [tile]: P_X of step g written (and O_X corrected)
    uint64_t *pv_done = p_full + kTiles;    // [tile]: PV_X of step g complete
    uint64_t *o_free = pv_done + kTiles;    // [tile]: the epilogue has read O_X (phase = X's blocks with work)
    uint64_t *final_bar = o_free + kTiles;  // every MMA of the CTA has completed
    // Windowed: a block's epilogue writes O into the one staging buffer, 64 columns at a time, and stores it by TMA.
    uint64_t *stage_full = final_bar + 1;   // the four softmax warps have written the buffer
    uint64_t *stage_free = stage_full + 1;  // the store before has finished reading it
    uint64_t *s_free = stage_free + 1;      // kOwnP: the softmax has loaded S of step g
    uint64_t *block_full = s_free + 1;              // [kBlocks]
    uint64_t *block_empty = block_full + kBlocks;   // [kBlocks]: every softmax warp has read it
    SoftBlock *soft_blocks = reinterpret_cast<SoftBlock *>(smem + L::kBlockOff);
    uint8_t *stage = smem + L::kStageOff;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + L::kTmemHolderOff);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_work = span_blocks<kTiles>(a, PREFIX);

    if (threadIdx.x == 0) {
        for (int b = 0; b < kQBufs; ++b) {
            mbar_init(&q_full[b], 1);
            mbar_init(&q_empty[b], 1);
        }
        for (int s = 0; s < NSLOT; ++s) {
            mbar_init(&slot_full[s], 1);
            mbar_init(&slot_empty[s], 1);
        }
        for (int x = 0; x < kTiles; ++x) {
            mbar_init(&s_full[x], 1);
            mbar_init(&p_full[x], 4);  // one arrive per softmax warp of tile x
            mbar_init(&pv_done[x], 1);
            mbar_init(&o_free[x], 4);
        }
        mbar_init(final_bar, 1);
        mbar_init(stage_full, 4);
        mbar_init(stage_free, 1);
        mbar_init(s_free, 4);
        for (int b = 0; b < kBlocks; ++b) {
            mbar_init(&block_full[b], 1);
            mbar_init(&block_empty[b], 4 * kTiles);
        }
        fence_mbarrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if constexpr (PREFIX) launch_dependents();
    const uint32_t tmem = *tmem_holder;

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            tma_prefetch_desc(&tmap_q);
            tma_prefetch_desc(&tmap_k);
            tma_prefetch_desc(&tmap_v);
            int last_round[NSLOT];
#pragma unroll
            for (int s = 0; s < NSLOT; ++s) last_round[s] = -1;
            int gidx = 0;  // K/V loads so far (ring position)
            int nb = 0;    // blocks so far
            bool ok = true;
            auto publish = [&](const SoftBlock *sb) {  // block nb (or the end) for the softmax warps
                const int e = nb % kBlocks;
                if (nb >= kBlocks && !mbar_wait(&block_empty[e], (nb / kBlocks - 1) & 1, a.status, kSiteBlock)) return false;
#pragma unroll
                for (int x = 0; x < kTiles; ++x) soft_blocks[e * kTiles + x] = sb[x];
                mbar_arrive(&block_full[e]);  // release: the entry is visible to the warps that wait on this phase
                return true;
            };
            for (int k = 0; ok && k * (int)gridDim.x < n_work; ++k) {
                const int Lw = persistent_work_index(k, n_work);
                if (Lw < 0) continue;
                const SpanBlock<kTiles> w = span_block<PREFIX, kTiles, kBN>(a, Lw);
                SoftBlock sb[kTiles];
#pragma unroll
                for (int x = 0; x < kTiles; ++x)
                    sb[x] = SoftBlock{w.n[x], w.span.n_sink, w.y_off + w.span.lo, nb, w.zq[x], w.yq[x], w.p0[x], w.kv_bh};
                if (!(ok = publish(sb))) break;
                // Q of this block goes after its first K and V tiles: its buffer frees only when the
                // previous block's last S products complete, and K_0 / V_0 need not wait for that
                // (a second buffer has been free since the block before that)
                const int q_at = nb < kQBufs || kQBufs == 2 ? 0 : 2;
                const int qb = nb % kQBufs;
                uint8_t *q_dst = q_s + qb * kTiles * L::kQBytes;
                for (int idx = 0; ok && idx <= 2 * w.span.n; ++idx) {
                    if (idx == q_at) {
                        if (nb >= kQBufs && !(ok = mbar_wait(&q_empty[qb], (nb / kQBufs - 1) & 1, a.status, kSiteQEmpty)))
                            break;
                        const int n_q_tiles = kTiles == 2 && w.n[kTiles - 1] > 0 ? 2 : 1;
                        if constexpr (PREFIX) {
                            // rb rows of each of nb sequences, packed; the tile's rows behind them keep
                            // whatever was there (no row's result depends on another row, and they are
                            // not stored)
                            mbar_arrive_expect_tx(&q_full[qb], n_q_tiles * a.parts.rb * a.parts.nb * D * 2);
                            for (int x = 0; x < n_q_tiles; ++x) {
                                int b0, r0;
                                packed_tile(a, w.yq[x], &b0, &r0);
#pragma unroll
                                for (int p = 0; p < kPanels; ++p)
                                    tma_load_4d(q_dst + x * L::kQBytes + p * (kBM * 128), &tmap_q, &q_full[qb], p * 64, r0,
                                                w.kv_bh, b0);
                            }
                        } else {
                            mbar_arrive_expect_tx(&q_full[qb], n_q_tiles * L::kQBytes);
                            for (int x = 0; x < n_q_tiles; ++x)
#pragma unroll
                                for (int p = 0; p < kPanels; ++p)
                                    tma_load_3d(q_dst + x * L::kQBytes + p * (kBM * 128), &tmap_q, &q_full[qb], p * 64,
                                                w.yq[x], w.zq[x]);
                        }
                    }
                    if (idx == 2 * w.span.n) break;
                    const int g = gidx + idx;
                    const int slot = g % NSLOT, round = g / NSLOT;
                    if (!(ok = mbar_wait(&slot_empty[slot], (round & 1) ^ 1, a.status, kSiteSlotEmpty))) break;
                    uint8_t *dst = slots + slot * L::kSlotBytes;
                    // a sink tile reads keys past the last sink as zeros (its maps end there): whatever the
                    // rows between the sinks and the window hold cannot reach a product
                    const int j = idx >> 1;
                    const bool sink = j < w.span.n_sink;
                    const CUtensorMap *map = (idx & 1) ? (sink ? &tmap_vs : &tmap_v) : (sink ? &tmap_ks : &tmap_k);
                    mbar_arrive_expect_tx(&slot_full[slot], L::kSlotBytes);
#pragma unroll
                    for (int p = 0; p < kPanels; ++p)
                        tma_load_3d(dst + p * (kBN * 128), map, &slot_full[slot], p * 64,
                                    w.y_off + w.span.key0(j, kBN), w.kv_bh);
#pragma unroll
                    for (int s = 0; s < NSLOT; ++s)
                        if (s == slot) last_round[s] = round;
                }
                gidx += 2 * w.span.n;
                ++nb;
            }
            if (ok) {
                SoftBlock end[kTiles];
#pragma unroll
                for (int x = 0; x < kTiles; ++x) end[x] = SoftBlock{-1, 0, 0, 0, 0, 0, 0, 0};
                publish(end);
            }
            // Drain: never leave the CTA with a TMA write still in flight.
#pragma unroll
            for (int s = 0; s < NSLOT; ++s)
                if (last_round[s] >= 0) mbar_wait(&slot_full[s], last_round[s] & 1, a.status, kSiteDrain);
            for (int b = max(0, nb - kQBufs); b < nb; ++b)
                mbar_wait(&q_full[b % kQBufs], (b / kQBufs) & 1, a.status, kSiteDrain);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ the tcgen05 issuer
        // The whole warp runs the loop (operands stay warp-uniform); one elected lane issues the MMAs
        // and the commits that track them.  Per block the order is
        //   one tile   S(0) | S(j+1) PV(j) | ...
        //   two tiles  S_A(0) S_B(0) | PV_A(j) S_A(j+1) PV_B(j) S_B(j+1) | ...
        constexpr uint32_t idesc_s = idesc_bf16_f32(kBM, kBN, false, false), idesc_sink = idesc_bf16_f32(kBM, 32, false, false);
        constexpr uint32_t idesc_o = idesc_bf16_f32(kBM, D, false, true);
        const uint32_t slot_addr = smem_u32(slots);
        const bool leader = elect_one();
        bool ok = true;
        int gidx = 0;                 // ring position of this block's K_0
        int step0[kTiles] = {};   // steps of tile x before this block
        int blocks[kTiles] = {};  // earlier blocks in which tile x had work (epilogues)
        int nb = 0;
        for (int k = 0; ok && k * (int)gridDim.x < n_work; ++k) {
            const int Lw = persistent_work_index(k, n_work);
            if (Lw < 0) continue;
            const SpanBlock<kTiles> w = span_block<PREFIX, kTiles, kBN>(a, Lw);
            const int qb = nb % kQBufs;
            const uint64_t q_desc = sdesc_sw128(smem_u32(q_s + qb * kTiles * L::kQBytes), 16, 1024);
            if (!(ok = warp_wait(&q_full[qb], (nb / kQBufs) & 1, a.status, kSiteQ))) break;
            tc_fence_after();
            // S_X(j) = Q_X K_j^T into S_X
            auto issue_s = [&](int x, int j) {
                if (!ok || !w.reads(x, j)) return;
                const int g = gidx + 2 * j;
                const int slot = g % NSLOT;
                if (!(ok = warp_wait(&slot_full[slot], (g / NSLOT) & 1, a.status, kSiteSlotFull))) return;
                // S_X overwrites P_X of the step before (this block's or the previous one's); kOwnP: S itself, loaded by now
                const int st = step0[x] + j;
                if (st >= 1 && !(ok = warp_wait(kOwnP ? s_free : &pv_done[x], (st - 1) & 1, a.status,
                                                kOwnP ? kSiteSFree : kSitePV)))
                    return;
                tc_fence_after();
                const uint64_t k_desc = sdesc_sw128(slot_addr + slot * L::kSlotBytes, 16, 1024);
                if (leader) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t off = (ks >> 2) * (kBM * 128) + (ks & 3) * 32;
                        mma_ss(tmem + kColS + x * kBN, sdesc_add(q_desc, x * L::kQBytes + off),
                               sdesc_add(k_desc, (ks >> 2) * (kBN * 128) + (ks & 3) * 32),
                               tile_cols<PREFIX, kBN>(a, w.span.n_sink, j) == 32 ? idesc_sink : idesc_s, ks > 0);
                    }
                    mma_commit(&s_full[x]);
                }
                __syncwarp();
            };
            // O_X += P_X(j) V_j, P_X from TMEM
            auto issue_pv = [&](int x, int j) {
                if (!ok || !w.reads(x, j)) return;
                const int g = gidx + 2 * j + 1;
                const int slot = g % NSLOT;
                if (!(ok = warp_wait(&slot_full[slot], (g / NSLOT) & 1, a.status, kSiteSlotFull))) return;
                if (!(ok = warp_wait(&p_full[x], (step0[x] + j) & 1, a.status, kSitePFull))) return;
                // the first PV of a block overwrites O_X, which the previous block's epilogue reads
                const bool first = j == 0;
                if (first && blocks[x] >= 1 && !(ok = warp_wait(&o_free[x], (blocks[x] - 1) & 1, a.status, kSiteOFree)))
                    return;
                tc_fence_after();
                const uint64_t v_desc = sdesc_sw128(slot_addr + slot * L::kSlotBytes, kBN * 128, 1024);
                const int steps = tile_cols<PREFIX, kBN>(a, w.span.n_sink, j) / 16;
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < kBN / 16; ++kk)
                        if (kk < 2 || kk < steps) mma_ts(tmem + kColO + x * D, tmem + kColP + x * kBN + kk * 8, sdesc_add(v_desc, kk * 2048),
                               idesc_o, (!first || kk > 0));
                    mma_commit(&pv_done[x]);
                }
                __syncwarp();
            };
            // a slot is released by a commit after the last MMA that reads it (a commit tracks every
            // earlier MMA of this thread); the same goes for the Q buffer after the block's last S
            auto commit_to = [&](uint64_t *bar) {
                if (leader) mma_commit(bar);
                __syncwarp();
            };
            if constexpr (kOwnP) {
                for (int j = 0; ok && j <= w.span.n; ++j) {
                    if (j < w.span.n) {
                        issue_s(0, j);
                        if (ok && j + 1 == w.span.n) commit_to(&q_empty[qb]);
                        if (ok) commit_to(&slot_empty[(gidx + 2 * j) % NSLOT]);  // K_j
                    }
                    if (j > 0) {
                        issue_pv(0, j - 1);
                        if (ok) commit_to(&slot_empty[(gidx + 2 * j - 1) % NSLOT]);  // V_{j-1}
                    }
                }
            } else {
                issue_s(0, 0);
                issue_s(1, 0);
                if (ok && w.span.n == 1) commit_to(&q_empty[qb]);
                if (ok) commit_to(&slot_empty[gidx % NSLOT]);  // K_0
                for (int j = 0; ok && j < w.span.n; ++j) {
                    issue_pv(0, j);
                    issue_s(0, j + 1);
                    issue_pv(1, j);
                    if (ok) commit_to(&slot_empty[(gidx + 2 * j + 1) % NSLOT]);  // V_j
                    issue_s(1, j + 1);
                    if (ok && j + 2 == w.span.n) commit_to(&q_empty[qb]);  // the block's last S products
                    if (ok && j + 1 < w.span.n) commit_to(&slot_empty[(gidx + 2 * j + 2) % NSLOT]);  // K_{j+1}
                }
            }
#pragma unroll
            for (int x = 0; x < kTiles; ++x) {
                step0[x] += w.n[x];
                blocks[x] += w.n[x] > 0;
            }
            gidx += 2 * w.span.n;
            ++nb;
        }
        // every MMA complete: TMEM may be released
        if (leader) mma_commit(final_bar);
        __syncwarp();
        warp_wait(final_bar, 0, a.status, kSiteFinal);
    } else {
        // ------------------------------------------------------------ softmax / correction / epilogue
        const int x = (warp - kFirstSoftmaxWarp) >> 2;  // query tile of this warpgroup
        const int quarter = warp & 3;                   // TMEM lanes [32*quarter, 32*quarter + 32)
        const int r = quarter * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        const uint32_t s_col = kColS + x * kBN, o_col = kColO + x * D, p_col = kColP + x * kBN;
        const float c = a.scale_log2;
        bool ok = true;
        int step0 = 0;     // steps of this tile before the current block
        int stores = 0;    // windowed: stores of O so far (phase of stage_full)
        for (int k = 0; ok; ++k) {
            const int e = k % kBlocks;
            ok = mbar_wait(&block_full[e], (k / kBlocks) & 1, a.status, kSiteBlock);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            const SoftBlock w = soft_blocks[e * kTiles + x];
            warp_arrive(&block_empty[e]);
            if (w.n < 0) break;
            const int n = w.n, yq = w.yq, zq = w.zq, pos0 = w.p0;
            const int pos = pos0 + r;  // windowed: this row's position
            float m = -INFINITY, l = 0.f;  // running max (log2 units) and sum
            for (int step = 0; step < n; ++step) {
                // this S_X was issued after the step before's PV_X completed, so O_X and the P columns are free as well
                ok = mbar_wait(&s_full[x], (step0 + step) & 1, a.status, kSiteSFull);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                tc_fence_after();
                // Lazy correction: keep the stale max unless the row max grew by > 8 (factor 256).
                bool need;
                float m_base, alpha;
                auto new_max = [&](float mt) {
                    const float m_new = fmaxf(m, mt);
                    need = m_new > m + 8.f;
                    const float m_use = need ? m_new : m;
                    m_base = (m_use == -INFINITY) ? 0.f : m_use;
                    alpha = need ? ex2_approx(m - m_base) : 1.f;
                    m = m_use;
                };
                const uint64_t c2 = f2_pack(c, c);
                uint64_t nm2, acc2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
                // kOwnP: S is in registers, the next one may overwrite it; P is free, and O holds every earlier product, once
                // the step before's PV has completed.  (Otherwise this S was issued after that product.)
                auto s_loaded = [&] {
                    if constexpr (kOwnP) {
                        tc_fence_before();
                        warp_arrive(s_free);
                    }
                };
                auto p_free = [&] {
                    if constexpr (kOwnP) {
                        if (step0 + step >= 1) ok = mbar_wait(&pv_done[x], (step0 + step - 1) & 1, a.status, kSitePV);
                        ok = __all_sync(0xffffffffu, ok);
                        tc_fence_after();
                    }
                };
                // P = 2^(s c - m) of 32 keys as bf16 pairs over columns [16h, 16h + 16) of P_X; the scaling FMA and the
                // row sum run on fp32 pairs
                auto store_p = [&](const uint32_t *raw, int h) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint64_t y2 = f2_fma(f2_pack(__uint_as_float(raw[2 * i]), __uint_as_float(raw[2 * i + 1])), c2, nm2);
                        float y0, y1;
                        f2_unpack(y2, y0, y1);
                        const float p0 = ex2_approx(y0), p1 = ex2_approx(y1);
                        acc2[i & 1] = f2_add(acc2[i & 1], f2_pack(p0, p1));
                        pk[i] = pack_bf16x2(p0, p1);
                    }
                    tmem_st16(tmem + lane_base + p_col + h * 16, pk);
                };
                if (tile_cols<PREFIX, kBN>(a, w.n_sink, step) == 32) {
                    // a sink tile whose sinks fit into 32 columns: every row of the query tile sees all of them
                    uint32_t raw[32];
                    tmem_ld32(tmem + lane_base + s_col, raw);
                    tmem_wait_ld();
                    s_loaded();
                    const int left = a.sinks - step * kBN;
                    float mx = -INFINITY;
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        if (e >= left) raw[e] = 0xff800000u;  // -inf
                        mx = fmaxf(mx, __uint_as_float(raw[e]));
                    }
                    new_max(c * mx);
                    nm2 = f2_pack(-m_base, -m_base);
                    p_free();
                    if (kOwnP && !ok) break;
                    store_p(raw, 0);
                } else {
                    const bool sink = step < w.n_sink;
                    const int key0 = sink ? step * kBN : w.key0 + (step - w.n_sink) * kBN;
                    const int window = sink ? 0 : a.window;
                    uint32_t raw[kBN];
#pragma unroll
                    for (int ch = 0; ch < kBN / 32; ++ch) tmem_ld32(tmem + lane_base + s_col + ch * 32, raw + ch * 32);
                    tmem_wait_ld();
                    s_loaded();
                    bool unseen = false;  // this row sees none of the tile's keys
                    if (PREFIX ? key0 + kBN > a.Nk
                               : !all_seen(pos0 + 32 * quarter, pos0 + 32 * quarter + 31, key0, key0 + kBN - 1, window, a.sinks)) {
                        // s = min(s, bound): bound is a NaN where the key is seen (a minimum ignores it, so s stays,
                        // be it a NaN itself) and -inf where it is not (whatever s is, a NaN too).  A bound is one
                        // byte permutation that spreads a mask bit's sign; selecting by predicates took 900-1300 cycles
                        // more per 128 x 128 tile, a third of an unmasked one.
                        uint32_t any = 0;
#pragma unroll
                        for (int h = 0; h < kBN / 32; ++h) {
                            const uint32_t seen = PREFIX ? low_bits(a.Nk - key0 - 32 * h)
                                                         : seen_keys(pos, key0 + 32 * h, window, a.sinks);
                            any |= seen;
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const uint32_t w8 = seen << (7 - k);
#pragma unroll
                                for (int y = 0; y < 4; ++y) {
                                    uint32_t bound;
                                    asm("prmt.b32 %0, %1, %2, %3;"
                                        : "=r"(bound)
                                        : "r"(w8), "r"(0xff800000u), "r"(0x7600u + (8u + y) * 0x11u));
                                    uint32_t &s = raw[32 * h + 8 * y + k];
                                    s = __float_as_uint(fminf(__uint_as_float(s), __uint_as_float(bound)));
                                }
                            }
                        }
                        unseen = any == 0;
                    }
                    // row max of the raw scores (scale > 0 commutes with max): four chains of three-input maxima
                    float mx[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) mx[u] = __uint_as_float(raw[u]);
#pragma unroll
                    for (int i = 4; i + 8 <= kBN; i += 8)
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            mx[u] = fmax3(mx[u], __uint_as_float(raw[i + 2 * u]), __uint_as_float(raw[i + 2 * u + 1]));
#pragma unroll
                    for (int u = 0; u < 4; ++u) mx[u] = fmaxf(mx[u], __uint_as_float(raw[kBN - 4 + u]));
                    const float mt = fmax3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
                    new_max(unseen ? -INFINITY : c * mt);
                    nm2 = f2_pack(-m_base, -m_base);
                    p_free();
                    if (kOwnP && !ok) break;
#pragma unroll
                    for (int h = 0; h < kBN / 32; ++h) store_p(raw + 32 * h, h);
                }
                float r0, r1, r2, r3;
                f2_unpack(acc2[0], r0, r1);
                f2_unpack(acc2[1], r2, r3);
                l = l * alpha + ((r0 + r1) + (r2 + r3));
                if (step >= 1 && __any_sync(0xffffffffu, need)) {
                    uint32_t ov[32];
#pragma unroll
                    for (int ch = 0; ch < D / 32; ++ch) {
                        tmem_ld32(tmem + lane_base + o_col + ch * 32, ov);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                        tmem_st32(tmem + lane_base + o_col + ch * 32, ov);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(&p_full[x]);
            }
            if (!ok || n == 0) continue;
            // the block's last PV_X has completed: O_X is final
            step0 += n;
            ok = mbar_wait(&pv_done[x], (step0 - 1) & 1, a.status, kSiteFinal);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            tc_fence_after();
            uint32_t ov[32];
            if constexpr (PREFIX) {
                // this chunk's partial of the row: O unnormalised, m (log2 units) and l
                // (rows of the tile behind its packed ones are written too and never read)
                const size_t part = a.parts.at(w.kv_bh, yq) + zq;
                float *dst = a.parts.o + part * (kBM * D) + r * 8;
#pragma unroll
                for (int ch = 0; ch < D / 32; ++ch) {
                    tmem_ld32(tmem + lane_base + o_col + ch * 32, ov);
                    tmem_wait_ld();
                    if (ch == D / 32 - 1) {
                        tc_fence_before();
                        warp_arrive(&o_free[x]);
                    }
#pragma unroll
                    for (int v8 = 0; v8 < 4; ++v8) st_global_v8(dst + (ch * 4 + v8) * (kBM * 8), ov + 8 * v8);
                }
                // every score a NaN: m stays -inf, which would read as "sees nothing"
                a.parts.ml[part * kBM + r] = make_float2(l != l ? fmaxf(m, 0.f) : m, l);
            } else {
                const float inv_l = 1.f / l;
                if (yq + r < a.Nq) a.lse[(size_t)zq * a.Nq + yq + r] = (m + __log2f(l)) * 0.69314718055994531f;
                // O / l as bf16 through the staging buffer, kStageCols columns at a time: 128-byte-swizzled panels of 64
                // columns, row r of panel p at p * 16 KB + r * 128, its 16-byte chunk k at k ^ (r % 8) (conflict-free
                // across the lanes)
                constexpr int kParts = D / L::kStageCols, kPartPanels = L::kStageCols / 64;
                const bool storer = quarter == kFirstSoftmaxWarp % 4 && lane == 0;  // one thread stores
#pragma unroll
                for (int part = 0; part < kParts; ++part) {
                    const int use = w.use * kParts + part;
                    // the previous use's TMA store has finished reading the buffer (the thread that issued it waits for it
                    // only here)
                    if (use >= 1 && storer) {
                        tma_store_wait_read();
                        mbar_arrive(stage_free);
                    }
                    if (use >= 1) ok = mbar_wait(stage_free, (use - 1) & 1, a.status, kSiteStage);
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
#pragma unroll
                    for (int ch = 0; ch < L::kStageCols / 32; ++ch) {
                        tmem_ld32(tmem + lane_base + o_col + part * L::kStageCols + ch * 32, ov);
                        tmem_wait_ld();
                        if (part == kParts - 1 && ch == L::kStageCols / 32 - 1) {
                            // every read of O_X is done: the next block's first PV_X may overwrite it
                            tc_fence_before();
                            warp_arrive(&o_free[x]);
                        }
                        uint8_t *prow = stage + (ch >> 1) * (kBM * 128) + r * 128;
#pragma unroll
                        for (int v4 = 0; v4 < 4; ++v4)
                            st_shared_v4(prow + ((((ch & 1) * 4 + v4) ^ (r & 7)) << 4),
                                         pack_bf16x2(__uint_as_float(ov[v4 * 8 + 0]) * inv_l, __uint_as_float(ov[v4 * 8 + 1]) * inv_l),
                                         pack_bf16x2(__uint_as_float(ov[v4 * 8 + 2]) * inv_l, __uint_as_float(ov[v4 * 8 + 3]) * inv_l),
                                         pack_bf16x2(__uint_as_float(ov[v4 * 8 + 4]) * inv_l, __uint_as_float(ov[v4 * 8 + 5]) * inv_l),
                                         pack_bf16x2(__uint_as_float(ov[v4 * 8 + 6]) * inv_l, __uint_as_float(ov[v4 * 8 + 7]) * inv_l));
                    }
                    fence_proxy_async_smem();  // the staged tile is read by the TMA (async proxy)
                    warp_arrive(stage_full);
                    if (storer) {
                        // rows past Nq and columns past the caller's D are clipped by the tensor map
                        if (mbar_wait(stage_full, stores & 1, a.status, kSiteStage)) {
#pragma unroll
                            for (int p = 0; p < kPartPanels; ++p) {
                                const int col = part * L::kStageCols + p * 64;
                                if (col < a.D) tma_store_3d(&tmap_o, stage + p * (kBM * 128), col, yq, zq);
                            }
                            tma_store_commit();
                        } else {
                            ok = false;
                        }
                    }
                    ++stores;
                }
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            }
        }
        tma_store_wait_read();  // the CTA's shared memory must outlive the stores' reads
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D, int NSLOT, bool PREFIX, int kTiles = 2, int kCtas = 1, int kBN = 128>
cudaError_t launch_spec(const SpanArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                        const CUtensorMap &tks, const CUtensorMap &tvs, const CUtensorMap &to, cudaStream_t s) {
    using L = SpanSmem<D, NSLOT, kTiles, kBN>;
    static_assert(L::kAlloc <= 233472 / kCtas - 1024, "shared memory budget (a CTA's own, and 1 KB that the system takes)");
    auto kern = win_fwd_kernel<D, NSLOT, PREFIX, kTiles, kCtas, kBN>;
    static std::atomic<unsigned long long> allowed{0};
    cudaError_t e = allow_smem((const void *)kern, L::kAlloc, allowed);
    if (e != cudaSuccess) return e;
    const int n_work = span_blocks<kTiles>(a, PREFIX);
    const int ctas = (a.num_sms > 0 ? a.num_sms : kNumSms) * kCtas;
    kern<<<n_work < ctas ? n_work : ctas, L::kThreads, L::kAlloc, s>>>(tq, tk, tv, tks, tvs, to, a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_win_fwd(const SpanArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                           const CUtensorMap &tks, const CUtensorMap &tvs, const CUtensorMap &to, cudaStream_t s) {
    const bool prefix = a.parts.o != nullptr;
    switch (kernel_head_dim(a.D)) {
        case 64:
            return prefix ? launch_spec<64, 4, true>(a, tq, tk, tv, tks, tvs, to, s)
                          : launch_spec<64, 4, false, 1, 2>(a, tq, tk, tv, tks, tvs, to, s);
        case 128:
            return prefix ? launch_spec<128, 4, true>(a, tq, tk, tv, tks, tvs, to, s)
                          : launch_spec<128, 4, false, 1, 2, 64>(a, tq, tk, tv, tks, tvs, to, s);
        default: return launch_win_fwd_wide(a, tq, tk, tv, tks, tvs, s);
    }
}

}  // namespace fa
