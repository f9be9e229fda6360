// win_decode.cu -- attention of a few new rows per sequence against that
// sequence's cache, grouped heads: the serving form of windowed attention, and
// (window = everything, no sinks) the sequences' own part of shared-prefix decode.
//
// Rows: R = (Hq / Hkv) n_q rows of a sequence share a key head; row i of the n_q
// sits at position len - n_q + i of a sequence that holds len keys and sees key j
// iff j <= p and (j < sinks or j > p - window).  Per row the online softmax
// (base 2), O = sum_j P_j v_j / l, L = (m + log2 l) ln 2; a row that sees nothing
// gets O = 0, L = -inf.
//
// What bounds it: HBM.  Every cached row is read once for all R rows, R <= 16
// rows a CTA (more rows take more CTAs, which share the tiles through L2); at 16
// rows a byte of K or V feeds 16 multiply-adds, 4x what the FMA pipe does in the
// time the byte takes (64 sequences of 900 to 16384 keys, window 4096, 32/8 heads of
// 128: 147 us, 6.7 TB/s), so the products run on the tensor cores: 16 rows x 8 keys x 16
// columns mma.sync (rows past R are zeros).  tcgen05 would need 128 rows.
//   warp 4     TMA producer: 64-key K and V tiles into a ring
//   warps 0-3  16 keys of every tile each, with a softmax state of their own
//              (no exchange inside the loop); the four states are joined at the end
// A sequence's tiles are dealt to `splits` CTAs by its own length (read on the
// device).  Few splits (win_decode_cluster) form a cluster that joins them through
// distributed shared memory; the partials of more are joined by win_join_kernel; with
// one split the CTA writes O and L itself.  Behind a shared prefix it is
// launched as that kernel's programmatic dependent, so it runs on the SMs that the
// prefix kernel leaves it and in its tail: the prefix is bound by its products, the
// caches by HBM.  When all of both fits on the GPU at once, each CTA waits for the
// prefix's partials and joins them itself; otherwise win_join_kernel does.
// Keys outside [0, len), between the sinks and the window, or past a sink tile's
// last sink may hold anything (a cache's unwritten rows): their scores are
// replaced and their V rows cleared before the products.
#include "fa_internal.h"
#include "sm100_ptx.cuh"
#include "launch.cuh"
#include "win_decode.cuh"
#include <algorithm>
#include <cmath>

namespace fa {
namespace {

constexpr int kWarps = 4;                 // compute warps
constexpr int kKeys = 16 * kWarps;        // keys per tile
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kRowTile = 16;              // rows per CTA

enum : int { kSiteEmpty = 201, kSiteFull, kSiteDrain };

constexpr int kCluster = 8;               // most CTAs of a cluster (the portable limit)

template <int D>
struct DecSmem {
    static constexpr int kTile = kKeys * D * 2;                 // one K or V tile
    static constexpr int kStages = D == 64 ? 4 : 3;
    static constexpr int kRing = kStages * 2 * kTile;
    static constexpr int kJoin = kWarps * kRowTile * (D + 4) * 4 + kWarps * kRowTile * 8;  // at the end, over the ring
    static constexpr int kShare = kRowTile * D * 4 + kRowTile * 8;  // behind it: the CTA's joined state, for its cluster
    static constexpr int kShareOff = (kJoin + 15) / 16 * 16;
    static_assert(kShareOff + kShare <= kRing, "in the ring's memory");
    static constexpr int kBarOff = kRing > kJoin ? kRing : (kJoin + 15) / 16 * 16;
    static constexpr int kAlloc = kBarOff + 2 * kStages * 8 + 1024;
};

template <int D>
__global__ void __launch_bounds__(kThreads)
    win_decode_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                      WinDecodeArgs a) {
    using L = DecSmem<D>;
    constexpr int kPanels = D / 64, kStages = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kBarOff);
    uint64_t *empty = full + kStages;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rt = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
    const int h = blockIdx.y, b = blockIdx.z;
    const int kv = b * a.Hkv + h;
    const int len = a.lens ? max(0, min(a.N, a.lens[b])) : a.N;
    // positions of the first and last new row; a sequence shorter than n_q has rows before its start
    const int p0 = max(0, len - a.n_q), p1 = len - 1;
    const KeySpan span = p1 >= 0 ? key_span(p0, p1, a.window, a.sinks, kKeys) : KeySpan{0, 0, 0};
    const int per = (span.n + a.splits - 1) / a.splits;
    const int t0 = min(span.n, split * per), t1 = min(span.n, t0 + per);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kWarps);
        }
        fence_mbarrier_init();
    }
    __syncthreads();

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    const int g = lane >> 2, tq = lane & 3;  // fragment row (and row + 8), column pair
    bool ok = true;

    if (warp == kWarps) {
        if (lane == 0) {
            tma_prefetch_desc(&tmap_k);
            tma_prefetch_desc(&tmap_v);
            for (int t = t0; t < t1; ++t) {
                const int i = t - t0, s = i % kStages, round = i / kStages;
                if (!mbar_wait(&empty[s], (round & 1) ^ 1, a.status, kSiteEmpty)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(&full[s], 2 * L::kTile);
                const int key0 = span.key0(t, kKeys);
#pragma unroll
                for (int p = 0; p < kPanels; ++p) {
                    tma_load_3d(smem + s * 2 * L::kTile + p * (kKeys * 128), &tmap_k, &full[s], p * 64, key0, kv);
                    tma_load_3d(smem + s * 2 * L::kTile + L::kTile + p * (kKeys * 128), &tmap_v, &full[s], p * 64, key0,
                                kv);
                }
            }
            // the loads of the last rounds have landed before the CTA reuses or leaves its shared memory
            const int n = t1 - t0;
            for (int i = max(0, n - kStages); i < n && ok; ++i)
                mbar_wait(&full[i % kStages], (i / kStages) & 1, a.status, kSiteDrain);
        }
    } else if (t0 < t1) {
        // Q fragments: rows g and g + 8 of this CTA's 16, columns in pairs
        uint32_t qf[D / 16][4];
        {
            const uint32_t *q0 = reinterpret_cast<const uint32_t *>(
                static_cast<const __nv_bfloat16 *>(a.q) + ((size_t)kv * a.R + rt * kRowTile + g) * D);
            const bool v0 = rt * kRowTile + g < a.R, v1 = rt * kRowTile + g + 8 < a.R;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                qf[kk][0] = v0 ? q0[8 * kk + tq] : 0u;
                qf[kk][1] = v1 ? q0[4 * D + 8 * kk + tq] : 0u;
                qf[kk][2] = v0 ? q0[8 * kk + 4 + tq] : 0u;
                qf[kk][3] = v1 ? q0[4 * D + 8 * kk + 4 + tq] : 0u;
            }
        }
        // position of rows g and g + 8 (rows past R: any; they are not stored)
        const int pos[2] = {len - a.n_q + (rt * kRowTile + g) % a.n_q, len - a.n_q + (rt * kRowTile + g + 8) % a.n_q};
        // ldmatrix addresses: lane l gives row (l % 8) of matrix l / 8.
        //   K (keys x columns): matrices (keys 0-7, cols 0-7), (keys 0-7, cols 8-15), (keys 8-15, ...) x 2
        //   V, transposed: matrices (keys 0-7, cols 0-7), (keys 8-15, cols 0-7), (keys 0-7, cols 8-15), ...
        const int mi = lane >> 3, mr = lane & 7;
        const uint32_t k_row = 16 * warp + mr + (mi >> 1) * 8, k_chunk = mi & 1;
        const uint32_t v_row = 16 * warp + mr + (mi & 1) * 8, v_chunk = mi >> 1;
        const uint32_t base = smem_u32(smem);
        for (int t = t0; t < t1; ++t) {
            const int i = t - t0, s = i % kStages;
            ok = mbar_wait(&full[s], (i / kStages) & 1, a.status, kSiteFull);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            const uint32_t ks = base + s * 2 * L::kTile, vs = ks + L::kTile;
            float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};  // keys 0-7, 8-15 of this warp's 16
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t kf[4];
                // 16-byte chunk c of row r of a 64-column panel sits at c ^ (r % 8)
                const uint32_t chunk = (kk & 3) * 2 + k_chunk;
                ldsm4(kf, ks + (kk >> 2) * (kKeys * 128) + k_row * 128 + ((chunk ^ (k_row & 7)) << 4));
                mma16816(sc[0], qf[kk], kf[0], kf[1]);
                mma16816(sc[1], qf[kk], kf[2], kf[3]);
            }
            const int key0 = span.key0(t, kKeys) + 16 * warp;
            const bool sink = t < span.n_sink;
            const int window = span.window_in(t, a.window);
            // every key of this warp's 16 exists, and every row sees it
            const bool plain = key0 + 16 <= len && all_seen(p0, p1, key0, key0 + 15, window, a.sinks);
            if (!plain) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t seen = seen_keys(pos[r], key0, window, a.sinks);
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (!((seen >> (8 * n + 2 * tq + e)) & 1u)) sc[n][2 * r + e] = -INFINITY;
                }
            }
            uint32_t pf[4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float mx = fmaxf(fmaxf(sc[0][2 * r], sc[0][2 * r + 1]), fmaxf(sc[1][2 * r], sc[1][2 * r + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float mt = mx * a.scale_log2;
                if (mt > m[r] + 8.f) {  // rescale only when the maximum grows by more than 2^8
                    const float alpha = ex2_approx(m[r] - mt);
                    l[r] *= alpha;
#pragma unroll
                    for (int d = 0; d < D / 8; ++d) {
                        o[d][2 * r] *= alpha;
                        o[d][2 * r + 1] *= alpha;
                    }
                    m[r] = mt;
                }
                const float mb = m[r] == -INFINITY ? 0.f : m[r];
                const float p00 = ex2_approx(fmaf(sc[0][2 * r], a.scale_log2, -mb));
                const float p01 = ex2_approx(fmaf(sc[0][2 * r + 1], a.scale_log2, -mb));
                const float p10 = ex2_approx(fmaf(sc[1][2 * r], a.scale_log2, -mb));
                const float p11 = ex2_approx(fmaf(sc[1][2 * r + 1], a.scale_log2, -mb));
                l[r] += (p00 + p01) + (p10 + p11);  // this lane's columns; the quad is added at the end
                // P is the bf16 operand of the second product (half a step: up to 2^-8 of a weight); l adds it unrounded
                pf[r] = pack_bf16x2(p00, p01);
                pf[2 + r] = pack_bf16x2(p10, p11);
            }
            // V rows that no row may see: cleared, so that 0 x (whatever they hold) cannot reach O
            uint32_t keep0 = ~0u, keep1 = ~0u;
            if (!plain) {
                const int lim = sink ? min(len, a.sinks) : len;
                const int k = key0 + 2 * tq;
                keep0 = (k < lim ? 0xffffu : 0u) | (k + 1 < lim ? 0xffff0000u : 0u);
                keep1 = (k + 8 < lim ? 0xffffu : 0u) | (k + 9 < lim ? 0xffff0000u : 0u);
            }
            __syncwarp();
#pragma unroll
            for (int dd = 0; dd < D / 16; ++dd) {
                uint32_t vf[4];
                const uint32_t chunk = (dd & 3) * 2 + v_chunk;
                ldsm4t(vf, vs + (dd >> 2) * (kKeys * 128) + v_row * 128 + ((chunk ^ (v_row & 7)) << 4));
                mma16816(o[2 * dd], pf, vf[0] & keep0, vf[1] & keep1);
                mma16816(o[2 * dd + 1], pf, vf[2] & keep0, vf[3] & keep1);
            }
            warp_arrive(&empty[s]);
        }
    }
    // add l over the quad's columns, then join the four warps' states through shared memory (the ring is free:
    // every tile has landed and been read)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
    __syncthreads();
    constexpr int kLd = D + 4;  // row stride in floats
    float *jo = reinterpret_cast<float *>(smem);
    float2 *jml = reinterpret_cast<float2 *>(jo + kWarps * kRowTile * kLd);
    if (warp < kWarps) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float *row = jo + (warp * kRowTile + g + 8 * r) * kLd;
#pragma unroll
            for (int d = 0; d < D / 8; ++d)
                *reinterpret_cast<float2 *>(row + 8 * d + 2 * tq) = make_float2(o[d][2 * r], o[d][2 * r + 1]);
            if (tq == 0) jml[warp * kRowTile + g + 8 * r] = make_float2(m[r], l[r]);
        }
    }
    __syncthreads();
    launch_dependents();
    if (a.behind && a.join) launch_dependent_wait();
    // four columns a thread; the rows of a group of 8 columns are neighbouring lanes, as they lie in the prefix's partials
    const int n_rows = min(kRowTile, a.R - rt * kRowTile);
    for (int idx = threadIdx.x; idx < n_rows * (D / 4); idx += kThreads) {
        const int r = (idx >> 1) % n_rows, c = (idx >> 1) / n_rows * 8 + (idx & 1) * 4;
        const int rr = rt * kRowTile + r;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, jml[w * kRowTile + r].x);
        const float Mb = M == -INFINITY ? 0.f : M;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float ls = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float2 ml = jml[w * kRowTile + r];
            const float f = ex2_approx(ml.x - Mb);
            const float4 v = *reinterpret_cast<const float4 *>(jo + (w * kRowTile + r) * kLd + c);
            ls = fmaf(ml.y, f, ls);
            acc.x = fmaf(v.x, f, acc.x);
            acc.y = fmaf(v.y, f, acc.y);
            acc.z = fmaf(v.z, f, acc.z);
            acc.w = fmaf(v.w, f, acc.w);
        }
        if (ls != ls) M = Mb;  // scores that are NaN leave m at -inf, which would read as "sees nothing"
        const size_t row = (size_t)kv * a.R + rr;
        if (a.cluster) {
            *reinterpret_cast<float4 *>(smem + L::kShareOff + (r * D + c) * 4) = acc;
            if (c == 0) *reinterpret_cast<float2 *>(smem + L::kShareOff + kRowTile * D * 4 + r * 8) = make_float2(M, ls);
        } else if (!a.join) {
            const size_t slot = row * a.splits + split;
            // a chunk that the row sees nothing of: m = -inf, l = 0, and its O is not read
            if (M != -INFINITY) *reinterpret_cast<float4 *>(a.part_o + slot * D + c) = acc;
            if (c == 0) a.part_ml[slot] = make_float2(M, ls);
        } else {
            if (a.parts.o) {
                int tile, r;
                a.parts.place(b, rr, &tile, &r);
                const size_t part = a.parts.at(h, tile);
                const float2 *ml = a.parts.ml + part * 128 + r;
                const float *po = a.parts.o + part * (128 * D) + (c >> 3) * (128 * 8) + r * 8 + (c & 7);
                float Mn = M;
                for (int s = 0; s < a.parts.splits; ++s) Mn = fmaxf(Mn, ml[s * 128].x);  // a prefix chunk's m is finite
                const float f0 = ex2_approx(M - Mn);
                ls *= f0;
                acc.x *= f0, acc.y *= f0, acc.z *= f0, acc.w *= f0;
                M = Mn;
#pragma unroll 8
                for (int s = 0; s < a.parts.splits; ++s) {
                    const float2 t = ml[s * 128];
                    const float f = ex2_approx(t.x - Mn);
                    const float4 v = *reinterpret_cast<const float4 *>(po + (size_t)s * (128 * D));
                    ls = fmaf(t.y, f, ls);
                    acc.x = fmaf(v.x, f, acc.x);
                    acc.y = fmaf(v.y, f, acc.y);
                    acc.z = fmaf(v.z, f, acc.z);
                    acc.w = fmaf(v.w, f, acc.w);
                }
            }
            const float inv = ls > 0.f ? 1.f / ls : 0.f;
            uint2 w;
            w.x = pack_bf16x2(acc.x * inv, acc.y * inv);
            w.y = pack_bf16x2(acc.z * inv, acc.w * inv);
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + row * D + c) = w;
            if (c == 0) a.lse[row] = (M + __log2f(ls)) * 0.69314718055994531f;
        }
    }
    if (a.cluster) {
        // Every CTA of the cluster joins a share of the columns from all of their states.
        cluster_sync();
        const uint32_t share = smem_u32(smem + L::kShareOff);
        for (int idx = split * kThreads + threadIdx.x; idx < n_rows * (D / 4); idx += a.splits * kThreads) {
            const int r = idx / (D / 4), c = idx % (D / 4) * 4;
            float2 ml[kCluster];
            float4 v[kCluster];
            float M = -INFINITY;
#pragma unroll
            for (int s = 0; s < kCluster; ++s) {
                ml[s] = make_float2(-INFINITY, 0.f);
                v[s] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (s >= a.splits) continue;
                ml[s] = ld_cluster_f2(map_to_cta(share + kRowTile * D * 4 + r * 8, s));
                v[s] = ld_cluster_f4(map_to_cta(share + (r * D + c) * 4, s));
                M = fmaxf(M, ml[s].x);
            }
            const float Mb = M == -INFINITY ? 0.f : M;
            float ls = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int s = 0; s < kCluster; ++s) {
                const float f = ex2_approx(ml[s].x - Mb);
                ls = fmaf(ml[s].y, f, ls);
                acc.x = fmaf(v[s].x, f, acc.x);
                acc.y = fmaf(v[s].y, f, acc.y);
                acc.z = fmaf(v[s].z, f, acc.z);
                acc.w = fmaf(v[s].w, f, acc.w);
            }
            const float inv = ls > 0.f ? 1.f / ls : 0.f;
            const size_t row = (size_t)kv * a.R + rt * kRowTile + r;
            uint2 w;
            w.x = pack_bf16x2(acc.x * inv, acc.y * inv);
            w.y = pack_bf16x2(acc.z * inv, acc.w * inv);
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + row * D + c) = w;
            if (c == 0) a.lse[row] = (M + __log2f(ls)) * 0.69314718055994531f;
        }
        cluster_sync();  // no CTA leaves while another reads its state
    }
    // This grid must not end before the one it runs behind: the join's launch waits for this one alone.  The CTA that
    // starts last waits, so that no other gives up its place on an SM.
    if (a.behind && !a.join && blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1 && blockIdx.z == gridDim.z - 1)
        launch_dependent_wait();
}

// One CTA joins the partials (the prefix's, then its own) of ROWS rows: M = max m_t, O = sum O_t 2^(m_t - M) / l.  A
// thread owns four columns of a row; the rows of a group of 8 columns are neighbouring lanes, as they lie in the
// prefix's partials.  The other threads take every kWays-th partial; the ways are added in order.  One row a CTA
// where there are few (2.4 us for 16 rows of 9 partials, against 4.5 with a warp per row); as many as its threads
// hold where there are many (one row a CTA took 30 us for 16384 rows of 8 partials, whose 32-byte pieces it fetched
// from as many lines).
template <int D, int ROWS>
__global__ void __launch_bounds__(128) win_join_kernel(WinDecodeArgs a, PrefixParts parts) {
    constexpr int kCols = D / 4, kWays = 128 / (kCols * ROWS);
    static_assert(kWays >= 1, "128 threads");
    __shared__ float4 sum[kWays][ROWS][kCols];
    __shared__ float2 stat[kWays][ROWS];
    const int way = threadIdx.x / (kCols * ROWS), in_way = threadIdx.x % (kCols * ROWS);
    const int sub = (in_way >> 1) % ROWS, c = (in_way >> 1) / ROWS * 2 + (in_way & 1);
    const size_t rows = (size_t)a.B * a.Hkv * a.R, at = (size_t)blockIdx.x * ROWS + sub;
    const size_t row = at < rows ? at : rows - 1;  // (a last CTA's extra rows repeat the last one and are not stored)
    const int P = parts.o ? parts.splits : 0, n = P + a.splits;
    const float2 *ml = nullptr;
    const float *po = nullptr;
    if (P > 0) {
        const unsigned per_seq = a.Hkv * a.R, b = (unsigned)row / per_seq;
        const int in = (int)((unsigned)row % per_seq), h = in / a.R;
        int tile, r;
        parts.place((int)b, in % a.R, &tile, &r);
        const size_t part = parts.at(h, tile);
        ml = parts.ml + part * 128 + r;
        po = parts.o + part * (128 * D) + (c >> 1) * (128 * 8) + r * 8 + (c & 1) * 4;
    }
    const float2 *ml_own = a.part_ml + row * a.splits;
    const float *po_own = a.part_o + row * a.splits * D + 4 * c;
    launch_dependent_wait();
    // online over this way's partials, eight loads in flight
    float M = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kBatch = 8;
    for (int s0 = way; s0 < n; s0 += kWays * kBatch) {
        float2 t[kBatch];
        float4 v[kBatch];
        float Mn = M;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int s = s0 + u * kWays;
            t[u] = make_float2(-INFINITY, 0.f);
            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (s >= n) continue;
            t[u] = s < P ? ml[s * 128] : ml_own[s - P];
            v[u] = *reinterpret_cast<const float4 *>(s < P ? po + (size_t)s * (128 * D) : po_own + (size_t)(s - P) * D);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) Mn = fmaxf(Mn, t[u].x);
        const float Mb = Mn == -INFINITY ? 0.f : Mn;
        const float f0 = ex2_approx(M - Mb);
        l *= f0;
        acc.x *= f0, acc.y *= f0, acc.z *= f0, acc.w *= f0;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (t[u].x == -INFINITY) continue;  // a chunk that this row sees nothing of: its O was not written
            const float f = ex2_approx(t[u].x - Mb);
            l = fmaf(t[u].y, f, l);
            acc.x = fmaf(v[u].x, f, acc.x);
            acc.y = fmaf(v[u].y, f, acc.y);
            acc.z = fmaf(v[u].z, f, acc.z);
            acc.w = fmaf(v[u].w, f, acc.w);
        }
        M = Mn;
    }
    sum[way][sub][c] = acc;
    if (c == 0) stat[way][sub] = make_float2(M, l);
    __syncthreads();
    if (way > 0 || at >= rows) return;
    float Mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWays; ++w) Mx = fmaxf(Mx, stat[w][sub].x);
    const float Mb = Mx == -INFINITY ? 0.f : Mx;
    l = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWays; ++w) {
        const float f = ex2_approx(stat[w][sub].x - Mb);
        const float4 v = sum[w][sub][c];
        l = fmaf(stat[w][sub].y, f, l);
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    uint2 w;
    w.x = pack_bf16x2(acc.x * inv, acc.y * inv);
    w.y = pack_bf16x2(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + row * D + 4 * c) = w;
    if (c == 0) a.lse[row] = (Mx + __log2f(l)) * 0.69314718055994531f;
}

template <int D>
cudaError_t launch_decode_d(const WinDecodeArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, cudaStream_t s) {
    auto kern = win_decode_kernel<D>;
    static std::atomic<unsigned long long> allowed{0};
    cudaError_t e = allow_smem((const void *)kern, DecSmem<D>::kAlloc, allowed);
    if (e != cudaSuccess) return e;
    const int row_tiles = (a.R + kRowTile - 1) / kRowTile;
    return launch_behind(kern, dim3(row_tiles * a.splits, a.Hkv, a.B), kThreads, DecSmem<D>::kAlloc, a.behind,
                         a.cluster ? a.splits : 1, s, tk, tv, a);
}

// CTAs an SM holds at once (shared memory: 65 KB at D = 64, 97 KB at 128, 193 KB at 256)
int ctas_per_sm(int D) { return D == 64 ? 3 : D == 128 ? 2 : 1; }

}  // namespace

int win_decode_sms(int B, int Hkv, int R, int splits, int D) {
    const long long ctas = (long long)B * Hkv * ((R + kRowTile - 1) / kRowTile) * splits;
    const long long sms = (ctas + ctas_per_sm(D) - 1) / ctas_per_sm(D);
    return sms < (1 << 20) ? (int)sms : 1 << 20;
}

int win_decode_splits(int B, int Hkv, int R, int tiles, int D, int num_sms) {
    // Enough CTAs for one full wave, none with less than two tiles: a split costs its CTA a pipeline fill and the
    // join a partial per row.
    const long long units = (long long)B * Hkv * ((R + kRowTile - 1) / kRowTile);
    const long long slots = (long long)(num_sms > 0 ? num_sms : kNumSms) * ctas_per_sm(D);
    long long sp = slots / units;
    if (sp > (tiles + 1) / 2) sp = (tiles + 1) / 2;
    const long long least = ((long long)tiles * (kKeys / kWarps) + kMaxSum - 1) / kMaxSum;  // a warp adds up 16 keys of a tile
    if (sp < least) sp = least;
    if (sp < 1) sp = 1;
    return (int)sp;
}

int win_decode_cluster(int splits, int tiles) {
    // A cluster saves the second launch (2 us of the host's time, 3 with the workspace) and is as fast on the device while
    // its CTAs get three tiles at most: one sequence of 4 key heads at D = 128, window 1000: 10.2 us (10.9 with the
    // second launch); window 2000: 12.3 (11.2); window 8000: 18.5 (14.3).
    if (splits < 2) return 0;
    return splits <= kCluster || tiles <= 3 * kCluster ? std::min(splits, kCluster) : 0;
}

int win_decode_tile_keys() { return kKeys; }

cudaError_t launch_win_decode(const WinDecodeArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, cudaStream_t s) {
    switch (a.D) {
        case 64: return launch_decode_d<64>(a, tk, tv, s);
        case 128: return launch_decode_d<128>(a, tk, tv, s);
        case 256: return launch_decode_d<256>(a, tk, tv, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_win_join(const WinDecodeArgs &a, const PrefixParts &parts, cudaStream_t s) {
    const long long rows = (long long)a.B * a.Hkv * a.R;
    const bool many = rows > 1024;
    const int per = many ? 128 / (a.D / 4) : 1;
    auto kern = a.D == 64    ? (many ? win_join_kernel<64, 8> : win_join_kernel<64, 1>)
                : a.D == 128 ? (many ? win_join_kernel<128, 4> : win_join_kernel<128, 1>)
                             : (many ? win_join_kernel<256, 2> : win_join_kernel<256, 1>);
    return launch_behind(kern, dim3((unsigned)((rows + per - 1) / per)), 128, 0, true, 1, s, a, parts);
}

}  // namespace fa
