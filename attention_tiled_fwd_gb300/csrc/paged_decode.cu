// paged_decode.cu -- attention of a few new rows per sequence against its bf16 pages, and the join of both decodes' partials.
//
// Row r of a key head's R = (Hq / Hkv) n_q sits at position len - n_q + r % n_q and sees key j iff j <= p and
// (j < sinks or j > p - window).  Online softmax in base 2, O = sum P v / l, L = (m + log2 l) ln 2; a row that sees nothing
// gets O = 0, L = -inf.
//
// What bounds it: HBM.  Every cached row is read once for up to 8 NT of the R rows.  The products run transposed on
// 16 x 8 x 16 mma.sync, S^T = K q^T and O^T = V^T P^T, with 16 keys (or channels) as the tall side: 8 rows cost one
// instruction where rows as the tall side would leave half of it empty.  tcgen05 would need 128 of them.
//   warp 4     producer: 64-key tiles of keys and values into a ring, a TMA box for every page and 64 columns; above D = 64 keys
//   (warp 5)   alone, and warp 5 values: a warp's copies go out 25 ns apart, 16 or 32 of them a tile where pages are small (one
//              sequence of 3001 keys in pages of 16, D = 128, a cluster: 1.5 us less than with one producer)
//   warps 0-3  units of 16 keys each, with a softmax state of their own, joined at a list's end
// The work is one list of tiles, sequence by sequence and head by head, cut into equal runs for a grid of one wave, however
// long the sequences are (lengths are read on the device).  A CTA writes O and L of what it holds whole; of what it shares
// with its neighbours it writes a partial, and paged_join_kernel adds those up.  Where there are few lists of few tiles (the rule
// is paged_grid's, fa_api.cu), the CTAs of a cluster share a list instead and join its partials through distributed shared memory.
// Measured: 64 sequences of 900 to 16384 keys of 8 heads of 128 (2.27 GB) 330 us, 6.9 TB/s, which is the rate of a copy (8192 keys of
// heads of 64: 168 us, 6.4 TB/s; of 256: 609 us, 7.1 TB/s); one sequence of 3001 keys of 4 heads 10.1 us as a cluster; cut into runs
// 8.9: the launch, the search (1 us), q (1 us), a first tile (1.5 us), the join (2.5 us).
//
// Keys that a row does not see may hold anything: their scores are replaced; values that no row sees are cleared before the
// product, and those that some rows see are kept from the others where they are not finite (0 times them would be NaN).
#include "fa_internal.h"
#include "launch.cuh"
#include "paged_decode.cuh"
#include <algorithm>

namespace fa {
namespace {

constexpr int kWarps = kDecodeWarps;
constexpr int kTile = kUnit * kWarps;  // keys

enum : int { kSiteEmpty = 301, kSiteFull, kSiteDrain };

template <int D>
struct Cfg {
    static constexpr int kProducers = D == 64 ? 1 : 2;  // warps that load; two: one for keys, one for values
    static constexpr int kThreads = 32 * (kWarps + kProducers);
    static constexpr int kHalf = kTile * 2 * D;                // bytes of the tile's keys, or of its values
    static constexpr int kStages = D == 64 ? 4 : 3;
    static constexpr int kCtas = D == 64 ? 3 : D == 128 ? 2 : 1;  // an SM
    static constexpr int kJoinOff = kStages * 2 * kHalf;
    static constexpr int kMlOff = kJoinOff + kWarps * kJoinCols * 8 * 4;
    static constexpr int kBarOff = kMlOff + kWarps * 8 * 8;
    static constexpr int kScanOff = kBarOff + 2 * kStages * 8;
    static constexpr int kAlloc = kScanOff + kScan + 1024;
};

// What a list costs besides its tiles, in tiles (its length, q, the join, the stores), so that runs of many lists end with the
// others: with 1 or 2 instead, 256 sequences of 1 to 300 keys took 6, 15 and 22 % longer at D = 64, 128 and 256; they take 27.4, 41.4 and
// 80.6 us now, 43, 58 and 59 % of the pages' bytes at the rate of a copy.
template <int D>
constexpr int kListCost = D == 64 ? 4 : 3;

// Two weights as operands of two products: the bf16 numbers below them, and what those leave, off by half a step, 2^-15 of a weight at
// most.  (One product with rounded weights, off by 2^-8, made O's error 1.4 times that of its own rounding.)  No part of a weight is 0:
// an infinite value times 0 would be NaN.
__device__ __forceinline__ void weight_parts(uint32_t &most, uint32_t &rest, float p0, float p1) {
    const uint32_t m0 = (max(__float_as_uint(p0), 1u) - 1u) & 0xffff0000u, m1 = (max(__float_as_uint(p1), 1u) - 1u) & 0xffff0000u;
    most = transpose8(m0 >> 16 | m1);
    rest = transpose8(pack_bf16x2(p0 - __uint_as_float(m0), p1 - __uint_as_float(m1)));
}
// o += the weighted values of a unit, in fp32 as such.  The tensor cores drop what lies 2^-25 below a sum's largest addend, which over
// a list's 2^21 keys a warp, two products each, would be 3 % of O if it stayed in one accumulator.
__device__ __forceinline__ void add_weighted(float (&o)[4], const uint32_t (&values)[4], const uint32_t (&most)[2], const uint32_t (&rest)[2]) {
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    mma16816(sum, values, rest[0], rest[1]);
    mma16816(sum, values, most[0], most[1]);
    f2_unpack(f2_add(f2_pack(o[0], o[1]), f2_pack(sum[0], sum[1])), o[0], o[1]);
    f2_unpack(f2_add(f2_pack(o[2], o[3]), f2_pack(sum[2], sum[3])), o[2], o[3]);
}

template <int D, int NT>
__global__ void __launch_bounds__(Cfg<D>::kThreads, Cfg<D>::kCtas)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                        PagedDecodeArgs a) {
    using C = Cfg<D>;
    constexpr int kRows = 8 * NT, kPanels = D / 64;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBarOff);
    uint64_t *empty = full + C::kStages;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], C::kProducers);
            mbar_init(&empty[s], kWarps);
        }
        fence_mbarrier_init();
    }
    // (the barriers in either stand behind the set-up too)
    Run<kListCost<D>> run = a.cluster ? cluster_run<kTile, kListCost<D>>(a, smem + C::kScanOff) : find_run<kTile, C::kThreads, kListCost<D>>(a, smem + C::kScanOff);
    launch_dependents();
    const int per_seq = a.pool.Hkv * a.row_tiles;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;

    if (warp >= kWarps) {
        // a box: 64 columns of the rows of a tile that a page holds; `half`: the boxes of a tile's keys, or of its values
        const int box_rows = min(1 << a.pool.shift, kTile), boxes = kTile / box_rows, half = boxes * kPanels;
        const uint32_t box_bytes = box_rows * 128;
        const bool value = C::kProducers == 2 ? warp > kWarps : lane >= half;
        const int box = lane % half / kPanels, panel = lane % kPanels;
        uint8_t *dst = smem + (value ? C::kHalf : 0) + panel * (kTile * 128) + box * box_rows * 128;
        if (lane == 0) {
            tma_prefetch_desc(&tmap_k);
            tma_prefetch_desc(&tmap_v);
        }
        long long loaded = 0;
        for (long long left = run.count; left > 0 && ok;) {
            const Tiles tiles = Tiles::of<kTile>(a, run.b);
            int t0, t1;
            run.part(tiles.n, left, &t0, &t1);
            const int h = run.u / a.row_tiles;
            // the lane's entry of the table for a tile, if it needs one: read three tiles ahead
            auto entry = [&](int t, int *k0) {
                *k0 = tiles.tile(t) * kTile + box * box_rows;
                return t < t1 && lane < half * (3 - C::kProducers) && *k0 < tiles.len && (*k0 + box_rows > tiles.lo || *k0 < a.sinks);
            };
            auto page_at = [&](int t) {
                int k0;
                return entry(t, &k0) ? a.pool.entry(run.b, k0) : -1;
            };
            int next[3] = {page_at(t0), page_at(t0 + 1), page_at(t0 + 2)};
            for (int t = t0; t < t1; ++t, ++loaded) {
                const int page = next[0];
                next[0] = next[1], next[1] = next[2], next[2] = page_at(t + 3);
                ok = sleepy_wait(&empty[stage], phase ^ 1, a.status, kSiteEmpty);
                if (!ok) break;
                int k0;
                const bool mine = entry(t, &k0);
                const uint32_t need = __ballot_sync(0xffffffffu, mine);
                if (lane == 0) mbar_arrive_expect_tx(&full[stage], __popc(need) * box_bytes);
                __syncwarp();
                if (mine) {
                    const bool there = (unsigned)page < (unsigned)a.pool.n_pages;
                    if (!there) record_failure(a.status, kErrPage, 0);
                    const int slice = there ? page * a.pool.Hkv + h : a.pool.n_pages * a.pool.Hkv;  // past the last: zeros
                    tma_load_3d(dst + stage * 2 * C::kHalf, value ? &tmap_v : &tmap_k, &full[stage], panel * 64,
                                k0 & ((1 << a.pool.shift) - 1), slice);
                }
                if (++stage == C::kStages) stage = 0, phase ^= 1;
            }
            left = run.next(tiles.n, left, per_seq);
        }
        // the last loads have landed before the CTA leaves
        const int last = (int)min((long long)C::kStages, loaded);
        for (int i = 0; i < last && ok; ++i) {
            if (--stage < 0) stage = C::kStages - 1, phase ^= 1;
            ok = sleepy_wait(&full[stage], phase, a.status, kSiteDrain);
        }
        if (a.cluster) {
            cluster_sync();
            cluster_sync();
        }
        return;
    }

    const int g = lane >> 2, tq = lane & 3;
    // ldmatrix addresses: lane l gives row l % 8 of matrix l / 8.  Keys: (keys 0-7, columns 0-7), (keys 8-15, columns 0-7), then
    // columns 8-15; values, transposed: (keys 0-7, columns 0-7), (keys 0-7, columns 8-15), then keys 8-15.
    const int mi = lane >> 3, mr = lane & 7;
    const uint32_t k_row = kUnit * warp + mr + (mi & 1) * 8, v_row = kUnit * warp + mr + (mi >> 1) * 8;
    int tail = -1, tail_rest = 0;
    for (long long left = run.count; left > 0;) {
        const Tiles tiles = Tiles::of<kTile>(a, run.b);
        int t0, t1;
        run.part(tiles.n, left, &t0, &t1);
        if (t0 == t1) {  // the run begins or ends in front of the list's first tile
            left = run.next(tiles.n, left, per_seq);
            continue;
        }
        const int h = run.u / a.row_tiles, row0 = run.u % a.row_tiles * kRows;
        const size_t first_row = ((size_t)run.b * a.pool.Hkv + h) * a.R + row0;
        const int p_first = max(0, tiles.len - a.n_q), p_last = tiles.len - 1;

        float m[NT][2], l[NT][2], o[NT][D / 16][4];
        auto position = [&](int r) { return tiles.len - a.n_q + (row0 + r) % a.n_q; };  // rows past R: any; they are not stored
        uint32_t qf[NT][D / 16][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) m[n][e] = kNone, l[n][e] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
            const bool there = row0 + 8 * n + g < a.R;
            const uint32_t *q = reinterpret_cast<const uint32_t *>(static_cast<const __nv_bfloat16 *>(a.q) + (first_row + 8 * n + g) * D);
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) qf[n][i][e] = there ? __ldg(q + 8 * i + 4 * e + tq) : 0u;
        }

        for (int t = t0; t < t1; ++t) {
            if (ok) ok = sleepy_wait(&full[stage], phase, a.status, kSiteFull);
            if (ok) {
                const uint32_t ks = smem_u32(smem) + stage * 2 * C::kHalf, vs = ks + C::kHalf;
                const int key0 = tiles.tile(t) * kTile + kUnit * warp;
                // every key of the unit exists, and every row sees it
                const bool plain = key0 + kUnit <= tiles.len && all_seen(p_first, p_last, key0, key0 + kUnit - 1, a.window, a.sinks);
                float sc[NT][4];  // S^T: keys g and g + 8, rows 2 tq and 2 tq + 1
#pragma unroll
                for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    uint32_t kf[4];  // 16-byte chunk c of row r of a 64-column panel sits at c ^ (r % 8)
                    const uint32_t chunk = (i & 3) * 2 + (mi >> 1);
                    ldsm4(kf, ks + (i >> 2) * (kTile * 128) + k_row * 128 + ((chunk ^ (k_row & 7)) << 4));
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma16816(sc[n], kf, qf[n][i][0], qf[n][i][1]);
                }
                if (!plain) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t seen = seen_keys(position(8 * n + 2 * tq + e), key0, a.window, a.sinks);
                            if (!(seen >> g & 1u)) sc[n][e] = -INFINITY;
                            if (!(seen >> (g + 8) & 1u)) sc[n][2 + e] = -INFINITY;
                        }
                }
                // the weights' logarithms; the maxima are taken again only when a weight would grow past 2^8 (products rounded as those
                // of the maxima are: unrounded, scores past 2^32 left weights that overflow)
                auto logs = [&](int n, int e) { return __fmul_rn(sc[n][e], a.scale_log2) - m[n][e & 1]; };
                bool grow = false;
#pragma unroll
                for (int n = 0; n < NT; ++n) grow |= fmaxf(fmax3(logs(n, 0), logs(n, 1), logs(n, 2)), logs(n, 3)) > 8.f;
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float mt = fmaxf(sc[n][e], sc[n][2 + e]) * a.scale_log2;
                            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 4));
                            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 8));
                            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
                            if (mt - m[n][e] > 8.f) {  // (the very test, in the same roundings)
                                const float alpha = ex2_approx(m[n][e] - mt);
                                l[n][e] *= alpha;
#pragma unroll
                                for (int i = 0; i < D / 16; ++i) o[n][i][e] *= alpha, o[n][i][2 + e] *= alpha;
                                m[n][e] = mt;
                            }
                        }
                }
                // P^T as the second product's operand, in two parts: row g, keys 2 tq and 2 tq + 1 (+ 8)
                uint32_t pb[NT][2], rest[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[e] = ex2_approx(logs(n, e));
                    // this lane's keys, not rounded; the others' are added at the end
                    l[n][0] += p[0] + p[2], l[n][1] += p[1] + p[3];
                    weight_parts(pb[n][0], rest[n][0], p[0], p[1]);
                    weight_parts(pb[n][1], rest[n][1], p[2], p[3]);
                }
                uint32_t keep[2] = {~0u, ~0u};
                if (!plain) keep_seen(keep, used_keys(tiles, key0, a.sinks), tq);
                auto values = [&](uint32_t(&vf)[4], int i, const uint32_t(&only)[2]) {
                    const uint32_t chunk = (i & 3) * 2 + (mi & 1);
                    ldsm4t(vf, vs + (i >> 2) * (kTile * 128) + v_row * 128 + ((chunk ^ (v_row & 7)) << 4));
                    if (!plain) vf[0] &= only[0], vf[1] &= only[0], vf[2] &= only[1], vf[3] &= only[1];
                };
                bool finite = true;
                if (!plain && a.n_q > 1) {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        uint32_t vf[4];
                        values(vf, i, keep);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            finite &= (vf[e] & 0x7f80u) != 0x7f80u && (vf[e] & 0x7f800000u) != 0x7f800000u;
                    }
                }
                if (__all_sync(0xffffffffu, finite)) {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        uint32_t vf[4];
                        values(vf, i, keep);
#pragma unroll
                        for (int n = 0; n < NT; ++n) add_weighted(o[n][i], vf, pb[n], rest[n]);
                    }
                } else {
                    // the rows of one position at a time, with the values of the keys that they see
#pragma unroll 1
                    for (int q = 0; q < a.n_q; ++q) {
                        const int p = tiles.len - a.n_q + q;
                        uint32_t only[2];
                        keep_seen(only, seen_keys(p, key0, a.window, a.sinks), tq);
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            uint32_t vf[4];
                            values(vf, i, only);
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                float sum[4] = {o[n][i][0], o[n][i][1], o[n][i][2], o[n][i][3]};
                                add_weighted(sum, vf, pb[n], rest[n]);
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (position(8 * n + 2 * tq + (e & 1)) == p) o[n][i][e] = sum[e];
                            }
                        }
                    }
                }
                warp_arrive(&empty[stage]);
            }
            if (++stage == C::kStages) stage = 0, phase ^= 1;
        }

        // O and L of a list that this CTA holds whole, else a partial: in its first slot what began in a CTA before this one, in
        // its second what goes on behind it
        const bool whole = t0 == 0 && t1 == tiles.n && !a.cluster;
        const size_t slot = a.cluster ? 0 : ((size_t)blockIdx.x * 2 + (t0 == 0)) * kRows;
        // (a cluster's in the ring, which has no more to hold)
        float *part_o = a.cluster ? reinterpret_cast<float *>(smem) : a.part_o;
        float2 *part_ml = a.cluster ? reinterpret_cast<float2 *>(smem + kRows * D * 4) : a.part_ml;
        if (t0 == 0 && !whole) {
            tail = run.b * per_seq + run.u;
            tail_rest = tiles.n - t1;
        }
        float *buf = reinterpret_cast<float *>(smem + C::kJoinOff);
        float2 *ml = reinterpret_cast<float2 *>(smem + C::kMlOff);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 4);
                l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 8);
                l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 16);
            }
            JoinedRow joined;
#pragma unroll
            for (int c = 0; c < D / kJoinCols; ++c) {
                sync_warps();  // the buffer is free
                if (c == 0 && g < 2) ml[8 * warp + 2 * tq + g] = make_float2(l[n][g & 1] == 0.f ? -INFINITY : m[n][g & 1], l[n][g & 1]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float *to = buf + warp * (kJoinCols * 8) + (16 * i + g) * 8 + 2 * tq;
                    const float *v = o[n][4 * c + i];
                    *reinterpret_cast<float2 *>(to) = make_float2(v[0], v[1]);
                    *reinterpret_cast<float2 *>(to + 64) = make_float2(v[2], v[3]);
                }
                sync_warps();
                if (c == 0) joined.read(ml);
                join_warps<D, 1>(a, part_o, part_ml, buf, joined, whole, slot, first_row, 8 * n, a.R - row0, kJoinCols * c, [](int ch) { return ch; });
            }
        }
        left = run.next(tiles.n, left, per_seq);
    }
    if (a.cluster) {
        join_cluster<D>(a, reinterpret_cast<const float *>(smem), reinterpret_cast<const float2 *>(smem + kRows * D * 4),
                        *reinterpret_cast<const int *>(smem + C::kScanOff), kRows);
        return;
    }
    if (a.tails && threadIdx.x == 0)
        a.tails[blockIdx.x] = make_int2(tail, tail < 0 ? 0 : parts_behind(a.cut, *reinterpret_cast<long long *>(smem + C::kScanOff + kAllOff), tail_rest));
}

// Adds up the partials of the list that goes on behind CTA blockIdx.x of the kernel before, if one does: the CTA's second
// slot and the first ones of the CTAs behind it.  One row a CTA; a thread owns four columns of every kWays-th partial.
template <int D, int THREADS>
__global__ void __launch_bounds__(THREADS) paged_join_kernel(PagedDecodeArgs a, int rows) {
    constexpr int kCols = D / 4, kWays = THREADS / kCols;
    __shared__ float4 sum[kWays][kCols];
    __shared__ float2 stat[kWays];
    const int way = threadIdx.x / kCols, c = threadIdx.x % kCols, r = blockIdx.y;
    launch_dependent_wait();
    const int2 tail = a.tails[blockIdx.x];
    if (tail.x < 0) return;
    const int row0 = tail.x % a.row_tiles * rows, bh = tail.x / a.row_tiles;
    if (row0 + r >= a.R) return;
    float M = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kBatch = 4;
    for (int s0 = way; s0 < tail.y; s0 += kWays * kBatch) {
        float2 t[kBatch];
        float4 v[kBatch];
        float Mn = M;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int s = s0 + u * kWays;
            t[u] = make_float2(-INFINITY, 0.f);
            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (s >= tail.y) continue;
            const size_t at = ((size_t)(blockIdx.x + s) * 2 + (s == 0)) * rows + r;
            t[u] = a.part_ml[at];
            v[u] = *reinterpret_cast<const float4 *>(a.part_o + at * D + 4 * c);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) Mn = fmaxf(Mn, t[u].x);
        const float Mb = Mn == -INFINITY ? 0.f : Mn;
        const float f0 = ex2_approx(M - Mb);
        l *= f0;
        acc.x *= f0, acc.y *= f0, acc.z *= f0, acc.w *= f0;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const float f = ex2_approx(t[u].x - Mb);
            l = fmaf(t[u].y, f, l);
            acc.x = fmaf(v[u].x, f, acc.x);
            acc.y = fmaf(v[u].y, f, acc.y);
            acc.z = fmaf(v[u].z, f, acc.z);
            acc.w = fmaf(v[u].w, f, acc.w);
        }
        M = Mn;
    }
    sum[way][c] = acc;
    if (c == 0) stat[way] = make_float2(M, l);
    __syncthreads();
    if (way > 0) return;
    float Mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWays; ++w) Mx = fmaxf(Mx, stat[w].x);
    const float Mb = Mx == -INFINITY ? 0.f : Mx;
    l = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWays; ++w) {
        const float f = ex2_approx(stat[w].x - Mb);
        const float4 v = sum[w][c];
        l = fmaf(stat[w].y, f, l);
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
    }
    const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
    const size_t row = (size_t)bh * a.R + row0 + r;
    uint2 w;
    w.x = pack_bf16x2(acc.x * inv, acc.y * inv);
    w.y = pack_bf16x2(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + row * D + 4 * c) = w;
    if (c == 0) a.lse[row] = (Mx + __log2f(l)) * 0.69314718055994531f;
}

template <int D, int NT>
cudaError_t launch_d(const PagedDecodeArgs &a, int ctas, const CUtensorMap &tk, const CUtensorMap &tv, cudaStream_t s) {
    auto kern = paged_decode_kernel<D, NT>;
    static std::atomic<unsigned long long> allowed{0};
    const cudaError_t e = allow_smem((const void *)kern, Cfg<D>::kAlloc, allowed);
    if (e != cudaSuccess) return e;
    return launch_behind(kern, dim3(ctas), Cfg<D>::kThreads, Cfg<D>::kAlloc, false, std::max(1, a.cluster), s, tk, tv, a);
}

}  // namespace

// 8 rows a CTA, or 16 where there are more: twice the products for half the reads.
// Clusters: a tile costs them what a warp's copies cost (25 ns each), so fewer tiles where the pages are small.
template <int D>
PagedPlan plan_d(int R, int page) {
    const int copies = 2 * (D / 64) * (kTile / std::min(page, kTile)) / Cfg<D>::kProducers;
    return PagedPlan{kTile, R > 8 ? 16 : 8, Cfg<D>::kCtas, copies <= 8 ? 6 : 4};
}
PagedPlan paged_plan(int R, int D, int page) {
    return D == 64 ? plan_d<64>(R, page) : D == 128 ? plan_d<128>(R, page) : plan_d<256>(R, page);
}

cudaError_t launch_paged_decode(const PagedDecodeArgs &a, int ctas, const CUtensorMap &tk, const CUtensorMap &tv, cudaStream_t s) {
    const bool two = a.R > 8;
    switch (a.D) {
        case 64: return two ? launch_d<64, 2>(a, ctas, tk, tv, s) : launch_d<64, 1>(a, ctas, tk, tv, s);
        case 128: return two ? launch_d<128, 2>(a, ctas, tk, tv, s) : launch_d<128, 1>(a, ctas, tk, tv, s);
        case 256: return two ? launch_d<256, 2>(a, ctas, tk, tv, s) : launch_d<256, 1>(a, ctas, tk, tv, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_paged_join(const PagedDecodeArgs &a, int ctas, int rows, cudaStream_t s) {
    // many partials a list: eight of them at a time (one sequence of 9000 keys of one head of 256: 13.1 us instead of 16.9 with two
    // at a time, of 128 11.7 instead of 13.1 with four)
    const bool many = ctas > 8ll * a.B * a.pool.Hkv * a.row_tiles;
    auto kern = a.D == 64 ? paged_join_kernel<64, 128>
                : a.D == 128 ? (many ? paged_join_kernel<128, 256> : paged_join_kernel<128, 128>)
                             : (many ? paged_join_kernel<256, 512> : paged_join_kernel<256, 128>);
    return launch_behind(kern, dim3(ctas, std::min(a.R, rows)), many ? 2 * a.D : 128, 0, true, 1, s, a, rows);
}

}  // namespace fa
