// paged_decode4.cu -- attention of a few new rows per sequence against its 4-bit pages (the mathematics, the list of tiles
// and the join of partials as in paged_decode.cu).
//
// What bounds it: HBM, if the codes become operands cheaply enough: at 4.5 bits a value an SM gets 42 values a clock.  So a
// code pair takes one instruction: its bits 0-3 of a half-word are the fp16 number code 2^-24, bits 4-7 are code 2^-20, so an
// AND makes an operand register of two of them; the powers go into q and into O's last factor.
// Keys: sum_c q_c s (code_c - 8) for 32 channels is s (the product with the codes); the -8 sum q go in as one more product of
// the scales.  q is scaled by a power of two a row so that fp16 holds its bf16 values.  Values: the weights are multiplied with
// each group's scales (fp16, one rounding of the weight and one of the product: 2^-11 each, an eighth of the output's own), and a product
// with ones adds up what 8 has to be taken of.  Weights carry 2^6 and scales a power of two that follows the tile's largest: where
// weights or products are subnormal in fp16 they are off by 2^-26 of that scale at most, beside the heaviest weight.  (Scales whose
// largest is outside 2^-4 .. 2 take a product each for it: 122 instead of 118 us.)
//
//   warp 4     producer: tiles of keys and values into a ring, a bulk copy for every page
//   warps 0-3  kUnits neighbouring units of 16 keys of every tile each
// Measured, 8 heads of 128: 48 sequences of 9000 to 32768 keys 198 us, 5.83 TB/s (86 % of a copy's rate), 64 of 900 to 16384 in pages of
// 16 122 us, 5.2 TB/s (77 %).  A steady run of tiles goes at 95 %, 55 % of the issue slots taken over a launch of 61 us; the rest is its
// start (5 us), the lists' ends (3 us each) and CTAs of an SM that do not end together.
// Not kept: a ring for every warp, filled by itself, leaves room for 16 warps that compute instead of 12, but the copies' integer work
// comes four times (170 us where this took 147, before other steps).
//
// Keys that a row does not see may hold anything: their scores are replaced, and their scales cleared before the product.
#include "fa_internal.h"
#include "launch.cuh"
#include "paged_decode.cuh"
#include <algorithm>
#include <cuda_fp16.h>

namespace fa {
namespace {

constexpr int kWarps = kDecodeWarps;
constexpr int kThreads = 32 * (kWarps + 1);
// The tensor cores drop what lies 2^-25 below a sum, n 2^-26 of a sum of n products at most.  O's accumulators hold sum P s code, and
// that and 8 sum P s are larger than O by the root of the number of keys and more: every kCentreKeys keys of a warp 8 sum P s is taken off.
// What is left loses 2^-13 of itself in kFoldKeys keys; then it is taken out and added up in fp32, in local memory.  With all of that at
// a list's end alone, errors beside the output's own rounding (1.65e-3) were 2.2e-3 for lists of 32768 keys, heads of 128, and O lost 1.6 % at
// 8 10^6; now they are 3.2e-4, from the weights' roundings, at any length.  48 sequences of 9000 to 32768: 198 us with 512 and 4096 keys,
// 197 with 512 or 1024 and 8192 (196.5 without any), 202 with all of it every 2048, 204 every 1024.
constexpr int kCentreKeys = 512, kFoldKeys = 8192;
constexpr int kLift = 6;  // weights carry 2^6, so they are 2^14 at most

enum : int { kSiteEmpty = 311, kSiteFull, kSiteDrain };

template <int D>
struct Cfg {
    static constexpr int kUnits = D < 256 ? 2 : 1;                       // of 16 keys, a warp and tile
    static constexpr int kTile = kWarps * kUnits * kUnit;                // keys
    static constexpr int kHalf = kTile * 9 * D / 16;                     // bytes of the tile's keys, or of its values
    static constexpr int kStages = D == 128 ? 3 : 4;
    static constexpr int kCtas = D == 64 ? 4 : D == 128 ? 3 : 2;         // an SM
    static constexpr int kJoinOff = kStages * 2 * kHalf;
    static constexpr int kMlOff = kJoinOff + kWarps * kJoinCols * 8 * 4;
    static constexpr int kBarOff = kMlOff + kWarps * 8 * 8;
    static constexpr int kScanOff = kBarOff + 2 * kStages * 8;
    static constexpr int kAlloc = kScanOff + kScan;
    static_assert(kHalf % 16 == 0 && kBarOff % 8 == 0, "bulk copies start on 16 bytes");
};

__device__ uint4 g_zero_units[Cfg<128>::kHalf / 16];  // what a page that the pool has not reads as
static_assert(Cfg<256>::kHalf <= Cfg<128>::kHalf && Cfg<64>::kHalf <= Cfg<128>::kHalf, "a box fits");

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same from zero.
__device__ __forceinline__ void mma_f16_new(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// N words from shared memory.
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], uint32_t at) {
    if constexpr (N == 1) {
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at) : "memory");
    } else if constexpr (N == 2) {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                         : "r"(at + 4 * i)
                         : "memory");
    }
}
// A lane's words of both halves of a unit's codes, group by group.
template <int D>
__device__ __forceinline__ void load_codes(uint32_t (&w)[2][D / 32], uint32_t unit, int lane) {
    using U = Unit4<D>;
    const uint32_t at = unit + 4 * U::kWide * lane;
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int g = 0; g < U::kGroups; g += U::kWide) {
            uint32_t v[U::kWide];
            load_words(v, at + 4 * U::word(half, g, 0));
#pragma unroll
            for (int i = 0; i < U::kWide; ++i) w[half][g + i] = v[i];
        }
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t max_h2(uint32_t a, uint32_t b) {  // of magnitudes; NaN gives way
    uint32_t d;
    asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ float2 unpack_h2(uint32_t a) { return __half22float2(*reinterpret_cast<const __half2 *>(&a)); }
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A list's q as the products take it, lane by lane: operands of row g (`there`: it exists), the groups' -8 sum q as an operand
// against the keys' scales, in two parts, and the factors that take the scores of rows 2 tq and 2 tq + 1 to log2 units.
template <int D>
__device__ __forceinline__ void prepare_q(const __nv_bfloat16 *q, bool there, float scale_log2, int lane, uint32_t (&qf)[D / 16][2],
                                          uint32_t (&less)[2], float (&f)[2]) {
    constexpr int kGroups = D / 32;
    const int tq = lane & 3;
    uint4 x[kGroups];
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
        x[j] = there ? __ldg(reinterpret_cast<const uint4 *>(q) + 4 * j + tq) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) most = max(most, max(w[i] << 16 & 0x7fff0000u, w[i] & 0x7fff0000u));
    }
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
    // the row's largest magnitude becomes 2^14 .. 2^15 (a row of zeros or of the smallest numbers: less)
    const int up = min(114, 14 - max(-100, (int)(most >> 23) - 127));
    const float by = __int_as_float((127 + up) << 23);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int shift = 24 - __shfl_sync(0xffffffffu, up, 4 * (2 * tq + e));  // the codes' 2^-24 too
        f[e] = scale_log2 * __int_as_float((127 + shift / 2) << 23) * __int_as_float((127 + shift - shift / 2) << 23);
        f[e] = fminf(fmaxf(f[e], 1.2e-38f), 3e38f);  // (above 0: -inf times it stays -inf; finite: a product of 0 stays 0)
    }
    uint32_t part[2][kGroups];  // fp16 of -8 2^-24 sum q, and of what that leaves
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
        const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
        float c[8], sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16) * by;
            if (i & 1) c[i] *= 0.0625f;
        }
        qf[2 * j][0] = pack_h2(c[0], c[4]), qf[2 * j][1] = pack_h2(c[1], c[5]);
        qf[2 * j + 1][0] = pack_h2(c[2], c[6]), qf[2 * j + 1][1] = pack_h2(c[3], c[7]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 even = unpack_h2(qf[2 * j + i][0]), odd = unpack_h2(qf[2 * j + i][1]);
            sum += (even.x + even.y) + 16.f * (odd.x + odd.y);
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum *= -0x1p-21f;
        const __half high = __float2half_rn(sum);
        part[0][j] = __half_as_ushort(high);
        part[1][j] = __half_as_ushort(__float2half_rn(sum - __half2float(high)));
    }
    // the operand's columns: the groups' first parts, then their second ones (lane tq: two columns of each eight)
    less[0] = less[1] = 0u;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const int at = i % (kGroups / 2), second = i / (kGroups / 2);
        const uint32_t two = part[second][2 * at] | part[second][2 * at + 1] << 16;
        if (tq == i % 4) less[i / 4] = two;
    }
}

// What a list costs besides its tiles, in tiles: with 2, 1 and 1 instead, 100 sequences of 100 to 3000 keys took 37, 57 and 109 us at
// D = 64, 128 and 256, with these 35, 49 and 88 (38, 54 and 60 % of the pages' bytes at the rate of a copy); 64 of 900 to 16384 76, 121 and
// 253, with these 76, 118 and 237.
template <int D>
constexpr int kListCost = D == 64 ? 4 : D == 128 ? 3 : 5;

template <int D>
__global__ void __launch_bounds__(kThreads, Cfg<D>::kCtas) paged_decode4_kernel(PagedDecodeArgs a) {
    using C = Cfg<D>;
    using U = Unit4<D>;
    constexpr int kCentre = kCentreKeys / (C::kUnits * kUnit), kFold = kFoldKeys / (C::kUnits * kUnit);  // tiles
    constexpr int kTile = C::kTile, kGroups = D / 32, kRows = 8, kStages = C::kStages;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBarOff), *empty = full + kStages;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kWarps);
        }
        fence_mbarrier_init();
    }
    // (the barriers in either stand behind the set-up too)
    Run<kListCost<D>> run = a.cluster ? cluster_run<kTile, kListCost<D>>(a, smem + C::kScanOff) : find_run<kTile, kThreads, kListCost<D>>(a, smem + C::kScanOff);
    launch_dependents();
    const int per_seq = a.pool.Hkv * a.row_tiles;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;

    if (warp == kWarps) {
        // a box: the rows of a tile that a page holds; a lane for each of keys and values
        const int box_rows = min(1 << a.pool.shift, kTile), boxes = kTile / box_rows;
        const uint32_t box_bytes = box_rows * (9 * D / 16), page_bytes = (9 * D / 16) << a.pool.shift;
        const uint64_t page_stride = (uint64_t)page_bytes * a.pool.Hkv;
        const bool value = lane >= boxes;
        const int row = lane % boxes * box_rows;  // of the tile
        const uint32_t dst = smem_u32(smem) + (value ? C::kHalf : 0) + row * (9 * D / 16);
        const uint8_t *pages = value ? a.pool.v : a.pool.k;
        long long loaded = 0;
        for (long long left = run.count; left > 0 && ok;) {
            const Tiles tiles = Tiles::of<kTile>(a, run.b);
            int t0, t1;
            run.part(tiles.n, left, &t0, &t1);
            const uint32_t head = run.u / a.row_tiles * page_bytes;
            // the lane's entry of the table for a tile, if it needs one: read three tiles ahead
            auto entry = [&](int t, int *k0) {
                *k0 = tiles.tile(t) * kTile + row;
                return t < t1 && lane < 2 * boxes && *k0 < tiles.len && (*k0 + box_rows > tiles.lo || *k0 < a.sinks);
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
                    const uint8_t *from = pages + (uint32_t)page * page_stride + head + (k0 & ((1 << a.pool.shift) - 1)) * (9 * D / 16);
                    if ((unsigned)page >= (unsigned)a.pool.n_pages) {
                        record_failure(a.status, kErrPage, 0);
                        from = reinterpret_cast<const uint8_t *>(g_zero_units);
                    }
                    bulk_load(dst + stage * 2 * C::kHalf, from, box_bytes, &full[stage]);
                }
                if (++stage == kStages) stage = 0, phase ^= 1;
            }
            left = run.next(tiles.n, left, per_seq);
        }
        // the last loads have landed before the CTA leaves
        const int last = (int)min((long long)kStages, loaded);
        for (int i = 0; i < last && ok; ++i) {
            if (--stage < 0) stage = kStages - 1, phase ^= 1;
            ok = sleepy_wait(&full[stage], phase, a.status, kSiteDrain);
        }
        if (a.cluster) {
            cluster_sync();
            cluster_sync();
        }
        return;
    }

    const int g = lane >> 2, tq = lane & 3;
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
        // spans of keys (D = 128: a warp's of a tile; else tiles: for D = 64 and 256 a warp's spans measured 2 and 3 % slower) all of which exist
        // and are in every row's window
        constexpr int kSpans = D == 128 ? kWarps : 1, kSpan = kTile / kSpans;
        const int p_first = max(0, tiles.len - a.n_q), past = tiles.len - 1 - a.window;
        const int plain0 = past < 0 ? 0 : past / kSpan + 1, plain1 = (p_first + 1) / kSpan;

        // off: the running maximum (log2 units) less kLift; kNone while a row has seen nothing
        float off[2], l[2], f[2], o[D / 16][4];
        auto position = [&](int r) { return tiles.len - a.n_q + (row0 + r) % a.n_q; };  // rows past R: any; they are not stored
        uint32_t qf[D / 16][2], less[2];
        float ones[kGroups / 2][4];  // sum P s of an even group, and of the odd one behind it
        int up = 0;  // scales are taken times 2^up
#pragma unroll
        for (int e = 0; e < 2; ++e) off[e] = kNone, l[e] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
#pragma unroll
        for (int j = 0; j < kGroups / 2; ++j) ones[j][0] = ones[j][1] = ones[j][2] = ones[j][3] = 0.f;
        prepare_q<D>(static_cast<const __nv_bfloat16 *>(a.q) + (first_row + g) * D, row0 + g < a.R, a.scale_log2, lane, qf, less, f);

        // O's sums of the keys before the last kFoldKeys, and `off` then: in local memory (the registers are taken)
        float4 held[D / 16];
        float held_off[2];
        asm volatile("" ::"l"(held), "l"(held_off) : "memory");
        for (int t = t0; t < t1;) {
            for (const int stop = min(t1, t + kCentre); t < stop; ++t) {
                const int tile = tiles.tile(t), key_warp = tile * kTile + warp * (C::kUnits * kUnit);
                const int span = kSpans == 1 ? tile : tile * kSpans + warp;
                const bool plain = span >= plain0 && span < plain1;
                const uint32_t ks = smem_u32(smem) + stage * 2 * C::kHalf + warp * (C::kUnits * U::kBytes), vs = ks + C::kHalf;
                float sc[C::kUnits][4];  // S^T of the warp's units: keys g and g + 8, rows 2 tq and 2 tq + 1
                if (ok) ok = sleepy_wait(&full[stage], phase, a.status, kSiteFull);  // (after a time-out: on whatever is there)
#pragma unroll
                for (int w = 0; w < C::kUnits; ++w) {
                    const int key0 = key_warp + w * kUnit;
                    const uint32_t at = ks + w * U::kBytes, scales = at + U::kCodes;
                    uint32_t code[2][kGroups], s2[2][kGroups / 2], by[4];
                    load_codes<D>(code, at, lane);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        load_words(s2[half], scales + 2 * U::k_scale(g + 8 * half, 0));
                        uint32_t two[1];
                        load_words(two, scales + 2 * U::k_scale(g + 8 * half, 2 * (tq % (kGroups / 2))));
                        by[half] = by[2 + half] = two[0];
                    }
                    mma_f16_new(sc[w], by, less[0], less[1]);
#pragma unroll
                    for (int j = 0; j < kGroups; ++j) {
                        uint32_t x[4], y[4];
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const uint32_t c = code[half][j], d = c >> 8;
                            x[half] = c & 0x000f000fu, x[2 + half] = c & 0x00f000f0u;
                            y[half] = d & 0x000f000fu, y[2 + half] = d & 0x00f000f0u;
                        }
                        const float2 sa = unpack_h2(s2[0][j / 2]), sb = unpack_h2(s2[1][j / 2]);
                        const float s_lo = j & 1 ? sa.y : sa.x, s_hi = j & 1 ? sb.y : sb.x;
                        float part[4];
                        mma_f16_new(part, x, qf[2 * j][0], qf[2 * j][1]);
                        mma_f16(part, y, qf[2 * j + 1][0], qf[2 * j + 1][1]);
                        sc[w][0] = fmaf(s_lo, part[0], sc[w][0]), sc[w][1] = fmaf(s_lo, part[1], sc[w][1]);
                        sc[w][2] = fmaf(s_hi, part[2], sc[w][2]), sc[w][3] = fmaf(s_hi, part[3], sc[w][3]);
                    }
                    if (!plain) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t seen = seen_keys(position(2 * tq + e), key0, a.window, a.sinks);
                            if (!(seen >> g & 1u)) sc[w][e] = -INFINITY;
                            if (!(seen >> (g + 8) & 1u)) sc[w][2 + e] = -INFINITY;
                        }
                    }
                }
                // scales of the values of keys 2 tq and 2 tq + 1 (+ 8)
                uint32_t s2[C::kUnits][2][kGroups], bits = 0;
#pragma unroll
                for (int w = 0; w < C::kUnits; ++w) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) load_words(s2[w][half], vs + w * U::kBytes + U::kCodes + 2 * U::v_scale(2 * tq + 8 * half, 0));
                    if (!plain) {
                        // 0 times whatever the scales are of keys that the lane's row g does not see must not reach O
                        const int key0 = key_warp + w * kUnit;
                        uint32_t keep[2];
                        keep_seen(keep, seen_keys(position(g), key0, a.window, a.sinks), tq);
#pragma unroll
                        for (int half = 0; half < 2; ++half)
#pragma unroll
                            for (int j = 0; j < kGroups; ++j) s2[w][half][j] &= keep[half];
                    }
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int j = 0; j < kGroups; ++j) bits |= s2[w][half][j];
                }
                // Products of weights with scales are fp16: scales below 2 2^-up do not overflow (nor does any at up = -14).  Below 2^-14 they
                // are off by 2^-25 whatever their size, so `up` follows the tile's largest scale down as well: it stays above 2^-4 2^-up.
                // For up = 0 two tests mostly do: 2 and more have bit 14, and any one of the scales is no more than the largest.
                const bool over = (bits & 0x40004000u) != 0, enough = ((s2[0][0][0] + 0x54005400u) & 0x80008000u) != 0;  // (2^-4 is 0x2c00)
                if (up != 0 || __any_sync(0xffffffffu, over) || !__any_sync(0xffffffffu, enough)) {
                    uint32_t most = 0;
#pragma unroll
                    for (int w = 0; w < C::kUnits; ++w)
#pragma unroll
                        for (int half = 0; half < 2; ++half)
#pragma unroll
                            for (int j = 0; j < kGroups; ++j) most = max_h2(most, s2[w][half][j]);
                    const float2 mh = unpack_h2(most);
                    const uint32_t all = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(mh.x, mh.y)));
                    const int size = (int)(all >> 23) - 127, to = max(-14, min(15, -size));  // 2^size: its power of two
                    if (all != 0 && (size + up > 0 || size + up < -4) && to != up) {
                        const float by = __int_as_float((127 + to - up) << 23);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
#pragma unroll
                            for (int j = 0; j < kGroups / 2; ++j) ones[j][e] *= by;
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) o[i][e] *= by;
                        }
                        up = to;
                    }
                    const uint32_t by = (uint32_t)(up + 15) * 0x04000400u;
#pragma unroll
                    for (int w = 0; w < C::kUnits; ++w)
#pragma unroll
                        for (int half = 0; half < 2; ++half)
#pragma unroll
                            for (int j = 0; j < kGroups; ++j) s2[w][half][j] = mul_h2(s2[w][half][j], by);
                }

                // the weights' logarithms; the maxima are taken again only when a weight would grow past 2^8 (products rounded as those
                // of the maxima are: unrounded, scores past 2^26 left weights that fp16 does not hold)
                bool grow = false;
                float lg[C::kUnits][4];
                auto logs = [&] {
#pragma unroll
                    for (int w = 0; w < C::kUnits; ++w)
#pragma unroll
                        for (int e = 0; e < 4; ++e) lg[w][e] = __fmul_rn(sc[w][e], f[e & 1]) - off[e & 1];
                };
                logs();
                constexpr float most = 8.f + kLift;
#pragma unroll
                for (int w = 0; w < C::kUnits; ++w)
                    grow |= fmaxf(fmax3(lg[w][0], lg[w][1], lg[w][2]), lg[w][3]) > most;
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mt = -INFINITY;
#pragma unroll
                        for (int w = 0; w < C::kUnits; ++w) mt = fmax3(mt, sc[w][e], sc[w][2 + e]);
                        mt *= f[e];
                        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 4));
                        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 8));
                        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
                        if (mt - off[e] > most) {  // (the very test, in the same roundings)
                            mt -= (float)kLift;
                            const float alpha = ex2_approx(off[e] - mt);
                            l[e] *= alpha;
#pragma unroll
                            for (int j = 0; j < kGroups / 2; ++j) ones[j][e] *= alpha, ones[j][2 + e] *= alpha;
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) o[i][e] *= alpha, o[i][2 + e] *= alpha;
                            off[e] = mt;
                        }
                    }
                    logs();
                }

#pragma unroll
                for (int w = 0; w < C::kUnits; ++w) {
                    const int key0 = key_warp + w * kUnit;
                    uint32_t pb[2];  // P^T as the second product's operand: row g, keys 2 tq and 2 tq + 1 (+ 8)
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[e] = ex2_approx(lg[w][e]);
                    // this lane's keys, not rounded; the others' are added at the end
                    l[0] += p[0] + p[2], l[1] += p[1] + p[3];
                    pb[0] = transpose8(pack_h2(p[0], p[1]));  // the weights as operands: fp16, off by 2^-11
                    pb[1] = transpose8(pack_h2(p[2], p[3]));
                    uint32_t code[2][kGroups];
                    load_codes<D>(code, vs + w * U::kBytes, lane);
#pragma unroll
                    for (int j = 0; j < kGroups; ++j) {
                        uint32_t x[4], y[4];
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const uint32_t c = code[half][j], d = c >> 8;
                            x[2 * half] = c & 0x000f000fu, x[2 * half + 1] = c & 0x00f000f0u;
                            y[2 * half] = d & 0x000f000fu, y[2 * half + 1] = d & 0x00f000f0u;
                        }
                        const uint32_t u0 = j & 1 ? 0u : 0x3c003c00u, u1 = 0x3c003c00u - u0, one[4] = {u0, u1, u0, u1};  // rows 0-7, or 8-15
                        const uint32_t b0 = mul_h2(pb[0], s2[w][0][j]), b1 = mul_h2(pb[1], s2[w][1][j]);
                        mma_f16(o[2 * j], x, b0, b1);
                        mma_f16(o[2 * j + 1], y, b0, b1);
                        mma_f16(ones[j / 2], one, b0, b1);
                    }
                }
                warp_arrive(&empty[stage]);
                if (++stage == kStages) stage = 0, phase ^= 1;
            }
            // 8 sum P s off the codes' sums
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const float *one = ones[i / 4] + (i & 2);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    o[i][e] = fmaf(one[e], -0x1p-21f, o[i][e]);
                    o[i][2 + e] = fmaf(one[e], -0x1p-17f, o[i][2 + e]);
                }
            }
#pragma unroll
            for (int j = 0; j < kGroups / 2; ++j) ones[j][0] = ones[j][1] = ones[j][2] = ones[j][3] = 0.f;
            if (t < t1 && (t - t0) % kFold != 0) continue;
            // O out of the accumulators, added up in fp32 as such
            const float by = __int_as_float((127 - up) << 23), by20 = 0x1p20f * by, by24 = 0x1p24f * by;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) o[i][0] *= by24, o[i][1] *= by24, o[i][2] *= by20, o[i][3] *= by20;
            if (t - t0 > kFold) {
                const float since0 = ex2_approx(held_off[0] - off[0]), since1 = ex2_approx(held_off[1] - off[1]);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const float4 h = held[i];
                    o[i][0] = fmaf(h.x, since0, o[i][0]);
                    o[i][1] = fmaf(h.y, since1, o[i][1]);
                    o[i][2] = fmaf(h.z, since0, o[i][2]);
                    o[i][3] = fmaf(h.w, since1, o[i][3]);
                }
            }
            if (t == t1) break;
            held_off[0] = off[0], held_off[1] = off[1];
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                held[i] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
                o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
            }
            asm volatile("" ::"l"(held), "l"(held_off) : "memory");
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
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 4);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 8);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 16);
        }
        JoinedRow joined;
#pragma unroll
        for (int c = 0; c < D / kJoinCols; ++c) {
            sync_warps();  // the buffer is free
            if (c == 0 && g < 2) ml[8 * warp + 2 * tq + g] = make_float2(l[g & 1] == 0.f ? -INFINITY : off[g & 1], l[g & 1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // channel 32 j + 4 g + (0, 1 | 2, 3) at place 8 (channel % 4) + g of its group
                const float *v = o[4 * c + i];
                float *to = buf + warp * (kJoinCols * 8) + (32 * (i / 2) + 16 * (i % 2) + g) * 8 + 2 * tq;
                *reinterpret_cast<float2 *>(to) = make_float2(v[0], v[1]);
                *reinterpret_cast<float2 *>(to + 64) = make_float2(v[2], v[3]);
            }
            sync_warps();
            if (c == 0) joined.read(ml);
            join_warps<D, 8>(a, part_o, part_ml, buf, joined, whole, slot, first_row, 0, a.R - row0, kJoinCols * c,
                             [](int ch) { return 32 * (ch / 32) + 8 * (ch % 4) + ch % 32 / 4; });
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

template <int D>
cudaError_t launch_d(const PagedDecodeArgs &a, int ctas, cudaStream_t s) {
    auto kern = paged_decode4_kernel<D>;
    static std::atomic<unsigned long long> allowed{0};
    const cudaError_t e = allow_smem((const void *)kern, Cfg<D>::kAlloc, allowed);
    if (e != cudaSuccess) return e;
    return launch_behind(kern, dim3(ctas), kThreads, Cfg<D>::kAlloc, false, std::max(1, a.cluster), s, a);
}

template <int D>
PagedPlan plan_d() {
    return PagedPlan{Cfg<D>::kTile, 8, Cfg<D>::kCtas, D < 256 ? 4 : 6};
}

}  // namespace

// 8 rows a CTA; more rows read the keys again.  (16 of them, with twice the accumulators, spill: 64 sequences of 8192, heads of 128
// took 251 us against 215 for two times 8, heads of 64 127 against 137.)
PagedPlan paged_plan4(int D) { return D == 64 ? plan_d<64>() : D == 128 ? plan_d<128>() : plan_d<256>(); }

cudaError_t launch_paged_decode4(const PagedDecodeArgs &a, int ctas, cudaStream_t s) {
    switch (a.D) {
        case 64: return launch_d<64>(a, ctas, s);
        case 128: return launch_d<128>(a, ctas, s);
        case 256: return launch_d<256>(a, ctas, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace fa
