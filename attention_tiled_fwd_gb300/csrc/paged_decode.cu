// paged_decode.cu -- attention of a few new rows per sequence against its pages, bf16 or 4-bit.
//
// Row r of a key head's R = (Hq / Hkv) n_q sits at position len - n_q + r % n_q and sees key j iff j <= p and
// (j < sinks or j > p - window).  Online softmax in base 2, O = sum P v / l, L = (m + log2 l) ln 2; a row that sees nothing
// gets O = 0, L = -inf.
//
// What bounds it: HBM.  Every cached row is read once for up to 8 NT of the R rows.  The products run transposed on
// 16 x 8 x 16 mma.sync, S^T = K q^T and O^T = V^T P^T, with 16 keys (or channels) as the tall side: 8 rows cost one
// instruction where rows as the tall side would leave half of it empty.  tcgen05 would need 128 of them.
//   warp 4     producer: tiles of keys and values into a ring (TMA boxes of bf16 pages, bulk copies of 4-bit units)
//   warps 0-3  units of 16 keys each, with a softmax state of their own, joined at a sequence's end
// The work is one list of tiles, sequence by sequence and head by head, cut into equal runs for a grid of one wave, however
// long the sequences are (lengths are read on the device).  A CTA writes O and L of what it holds whole; of what it shares
// with its neighbours it writes a partial, and paged_join_kernel adds those up.
//
// 4 bits: a code needs one instruction for two of them.  Its bits 0-3 of a half-word are the fp16 number code 2^-24, bits 4-7
// are code 2^-20, so an AND makes a pair of operands of them; the powers go into q and into O's last factor.
// Keys: sum_c q_c s (code_c - 8) for 32 channels is s (the product with the codes, begun at -8 sum q).  q is scaled by a power
// of two a row so that fp16 holds its bf16 values.  Values: the weights are multiplied with each group's scales (fp16, one
// rounding of the weight and one of the product: 2^-11 each), and a product with ones adds up what 8 has to be taken of.
// Weights carry a power of two, 2^-E, so that their products with the scales stay in fp16's range and above its subnormals: E
// grows with the scales.
//
// Keys that a row does not see may hold anything: their scores are replaced; values that no row sees are cleared before the
// product, and those that some rows see are kept from the others where they are not finite (0 times them would be NaN).
#include "fa_internal.h"
#include "launch.cuh"
#include "paged.cuh"
#include "sm100_ptx.cuh"
#include <algorithm>
#include <cuda_fp16.h>

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * (kWarps + 1);
constexpr float kNone = -3e38f;
constexpr int kTinyScales = -22;  // E while no scale has reached 2^-15: they are taken times 2^15, the weights times 2^7
constexpr int kJoinCols = 64;  // channels that the warps join at a time

enum : int { kSiteEmpty = 301, kSiteFull, kSiteDrain };

template <int D, int NT, bool FOUR>
struct Cfg {
    static constexpr int kTile = FOUR && D < 256 ? 128 : 64;                   // keys
    static constexpr int kUnits = kTile / kUnit / kWarps;                      // of 16 keys, a warp
    static constexpr int kRow = FOUR ? 9 * D / 16 : 2 * D;                     // bytes of a key
    static constexpr int kHalf = kTile * kRow;                                 // the tile's keys, or its values
    static constexpr int kStages = FOUR ? (D == 128 ? 3 : 4) : D == 64 ? 4 : 3;
    static constexpr int kCtas = FOUR ? (D == 64 ? (NT == 1 ? 4 : 3) : D == 128 && NT == 1 ? 3 : 2) : D == 64 ? 3 : D == 128 ? 2 : 1;  // an SM
    static constexpr int kJoinOff = kStages * 2 * kHalf;
    static constexpr int kMlOff = kJoinOff + kWarps * kJoinCols * 8 * 4;
    static constexpr int kBarOff = kMlOff + kWarps * 8 * 8;
    static constexpr int kScanOff = kBarOff + 2 * kStages * 8;
    static constexpr int kAlloc = kScanOff + 64 + 1024;
};

__device__ uint4 g_zero_units[128 * 72 / 16];  // what a page that the pool has not reads as (4-bit)

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
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
// The 8 x 8 matrix of 16-bit values that the warp holds, a row in four lanes, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
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

// Masks of the pairs of keys that a lane holds of a unit: 2 tq and 2 tq + 1, and 8 further; bit i of `seen`: key i.
__device__ __forceinline__ void keep_seen(uint32_t (&keep)[2], uint32_t seen, int tq) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const uint32_t two = seen >> (8 * half + 2 * tq);
        keep[half] = (two & 1u ? 0xffffu : 0u) | (two & 2u ? 0xffff0000u : 0u);
    }
}

// The tiles of a sequence: sink tiles from 0 on, then tiles from `first` on.
struct Tiles {
    int len, lo, n_sink, first, n;  // lo: the first key in any row's window
    template <int TILE>
    static __device__ __forceinline__ Tiles of(const PagedDecodeArgs &a, int b) {
        Tiles t;
        const int cap = a.pool.capacity();
        t.len = a.lens ? max(0, min(cap, __ldg(a.lens + b))) : cap;
        t.lo = max(0, max(0, t.len - a.n_q) - a.window + 1);
        const int sinks = (min(a.sinks, t.len) + TILE - 1) / TILE;
        const bool gap = t.lo / TILE > sinks;
        t.n_sink = gap ? sinks : 0;
        t.first = gap ? t.lo / TILE : 0;
        t.n = max(1, t.n_sink + (t.len + TILE - 1) / TILE - t.first);  // a sequence without keys has a tile that nobody sees
        return t;
    }
    __device__ __forceinline__ int tile(int i) const { return i < n_sink ? i : first + i - n_sink; }
};

// bit i: some row sees key k0 + i
__device__ __forceinline__ uint32_t used_keys(const Tiles &t, int k0, int sinks) {
    return low_bits(t.len - k0) & (~low_bits(t.lo - k0) | low_bits(sinks - k0));
}

// This CTA's run of the list of tiles.
struct Run {
    int b, u, t;      // sequence, key head and row tile, tile
    long long count;  // tiles
};

template <int TILE>
__device__ __forceinline__ long long tiles_of(const PagedDecodeArgs &a, int b0, int b1) {
    long long sum = 0;
    for (int b = b0; b < b1; ++b) sum += Tiles::of<TILE>(a, b).n;
    return sum;
}

// All threads: each adds up the tiles of its share of the sequences, and the one whose share the run begins in finds where.
template <int TILE>
__device__ __forceinline__ Run find_run(const PagedDecodeArgs &a, uint8_t *scratch) {
    long long *totals = reinterpret_cast<long long *>(scratch);
    int *where = reinterpret_cast<int *>(scratch + 8 * (kWarps + 1));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = (a.B + kThreads - 1) / kThreads, b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
    const long long mine = tiles_of<TILE>(a, b0, b1);
    long long before = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, before, d);
        if (lane >= d) before += x;
    }
    if (lane == 31) totals[warp] = before;
    before -= mine;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w <= kWarps; ++w) {
        if (w < warp) before += totals[w];
        total += totals[w];
    }
    const long long per_tile = (long long)a.pool.Hkv * a.row_tiles;
    const long long share = (total * per_tile + gridDim.x - 1) / gridDim.x, begin = share * blockIdx.x;
    Run r;
    r.count = min(share, total * per_tile - begin);
    if (begin >= before * per_tile && begin < (before + mine) * per_tile) {
        int b = b0;
        for (;; ++b) {
            const int n = Tiles::of<TILE>(a, b).n;
            if (begin < (before + n) * per_tile) {
                const long long in = begin - before * per_tile;
                where[0] = b, where[1] = (int)(in / n), where[2] = (int)(in % n);
                break;
            }
            before += n;
        }
    }
    __syncthreads();
    r.b = r.u = r.t = 0;
    if (r.count > 0) r.b = where[0], r.u = where[1], r.t = where[2];
    return r;
}

template <int D, int NT, bool FOUR>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT, FOUR>::kCtas)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                        PagedDecodeArgs a) {
    using C = Cfg<D, NT, FOUR>;
    using U = Unit4<D>;
    constexpr int kTile = C::kTile, kGroups = D / 32, kRows = 8 * NT;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBarOff);
    uint64_t *empty = full + C::kStages;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kWarps);
        }
        fence_mbarrier_init();
    }
    Run run = find_run<kTile>(a, smem + C::kScanOff);  // (its barriers stand behind the set-up too)
    launch_dependents();
    const int per_seq = a.pool.Hkv * a.row_tiles;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;

    if (warp == kWarps) {
        // a box: the rows of a tile that a page holds, or 64 columns of them
        const int box_rows = min(1 << a.pool.shift, kTile), boxes = kTile / box_rows;
        constexpr int kPanels = FOUR ? 1 : D / 64;
        const uint32_t box_bytes = box_rows * C::kRow / kPanels;
        const int copies = 2 * boxes * kPanels;
        const bool value = lane >= copies / 2;
        const int box = lane % (copies / 2) / kPanels, panel = lane % kPanels;
        uint8_t *dst = smem + (value ? C::kHalf : 0) + (FOUR ? box * box_bytes : panel * (kTile * 128) + box * box_rows * 128);
        if (!FOUR && lane == 0) {
            tma_prefetch_desc(&tmap_k);
            tma_prefetch_desc(&tmap_v);
        }
        long long left = run.count;
        for (; left > 0 && ok; ) {
            const Tiles tiles = Tiles::of<kTile>(a, run.b);
            const int t1 = (int)min((long long)tiles.n, run.t + left), h = run.u / a.row_tiles;
            // the lane's page of a tile, -1 where the pool has none; -2 where none is needed
            auto page_at = [&](int t) {
                const int k0 = tiles.tile(t) * kTile + box * box_rows;
                if (lane >= copies || k0 >= tiles.len || !(k0 + box_rows > tiles.lo || k0 < a.sinks)) return -2;
                return a.pool.page_of(run.b, k0);
            };
            int next = page_at(run.t);
            for (int t = run.t; t < t1; ++t) {
                const int page = next;
                if (t + 1 < t1) next = page_at(t + 1);
                ok = __all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1, a.status, kSiteEmpty));
                if (!ok) break;
                const uint32_t need = __ballot_sync(0xffffffffu, page != -2);
                if (lane == 0) mbar_arrive_expect_tx(&full[stage], __popc(need) * box_bytes);
                __syncwarp();
                if (page != -2) {
                    if (page == -1) record_failure(a.status, kErrPage, 0);
                    const int k0 = tiles.tile(t) * kTile + box * box_rows;
                    uint8_t *to = dst + stage * 2 * C::kHalf;
                    if constexpr (FOUR) {
                        const uint8_t *from = (value ? a.pool.v : a.pool.k) + a.pool.at(max(page, 0), h, k0, C::kRow);
                        bulk_load(to, page >= 0 ? from : reinterpret_cast<const uint8_t *>(g_zero_units), box_bytes, &full[stage]);
                    } else {
                        const int slice = page >= 0 ? page * a.pool.Hkv + h : a.pool.n_pages * a.pool.Hkv;  // past the last: zeros
                        tma_load_3d(to, value ? &tmap_v : &tmap_k, &full[stage], panel * 64, k0 & ((1 << a.pool.shift) - 1), slice);
                    }
                }
                if (++stage == C::kStages) stage = 0, phase ^= 1;
            }
            left -= t1 - run.t;
            run.t = 0;
            if (++run.u == per_seq) run.u = 0, ++run.b;
        }
        // the last loads have landed before the CTA leaves
        const int last = (int)min((long long)C::kStages, run.count);
        for (int i = 0; i < last && ok; ++i) {
            if (--stage < 0) stage = C::kStages - 1, phase ^= 1;
            ok = mbar_wait(&full[stage], phase, a.status, kSiteDrain);
        }
        return;
    }

    const int g = lane >> 2, tq = lane & 3;
    int tail = -1, tail_parts = 0;
    for (long long left = run.count; left > 0; ) {
        const Tiles tiles = Tiles::of<kTile>(a, run.b);
        const int t1 = (int)min((long long)tiles.n, run.t + left);
        const int h = run.u / a.row_tiles, row0 = run.u % a.row_tiles * kRows;
        const size_t first_row = ((size_t)run.b * a.pool.Hkv + h) * a.R + row0;
        const int p_first = max(0, tiles.len - a.n_q), p_last = tiles.len - 1;

        // off: the running maximum (log2 units), plus the weights' power of two; kNone while a row has seen nothing
        float off[NT][2], l[NT][2], f[NT][2], o[NT][D / 16][4];
        auto position = [&](int r) { return tiles.len - a.n_q + (row0 + r) % a.n_q; };  // rows past R: any; they are not stored
        uint32_t qf[NT][D / 16][2];
        uint32_t less[FOUR ? NT : 1][2];  // 4 bits: -8 sum q of each group as an operand against the keys' scales, in two parts
        float ones[FOUR ? NT : 1][4];     // sum P s of group g in row g
        int E = kTinyScales, Ep = FOUR ? -7 : 0;  // powers of two of the weights times scales, and of the weights
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) off[n][e] = kNone, l[n][e] = 0.f, f[n][e] = a.scale_log2;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
            const bool there = row0 + 8 * n + g < a.R;
            const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + (first_row + 8 * n + g) * D;
            if constexpr (!FOUR) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        qf[n][i][e] = there ? __ldg(reinterpret_cast<const uint32_t *>(q) + 8 * i + 4 * e + tq) : 0u;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) ones[n][e] = 0.f;
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
                    f[n][e] = fmaxf(a.scale_log2 * __int_as_float((127 + shift / 2) << 23) * __int_as_float((127 + shift - shift / 2) << 23),
                                    1.2e-38f);  // (above 0: -inf times it stays -inf)
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
                    qf[n][2 * j][0] = pack_h2(c[0], c[4]), qf[n][2 * j][1] = pack_h2(c[1], c[5]);
                    qf[n][2 * j + 1][0] = pack_h2(c[2], c[6]), qf[n][2 * j + 1][1] = pack_h2(c[3], c[7]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 even = unpack_h2(qf[n][2 * j + i][0]), odd = unpack_h2(qf[n][2 * j + i][1]);
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
                less[n][0] = less[n][1] = 0u;
#pragma unroll
                for (int i = 0; i < kGroups; ++i) {
                    const int at = i % (kGroups / 2), second = i / (kGroups / 2);
                    const uint32_t two = part[second][2 * at] | part[second][2 * at + 1] << 16;
                    if (tq == i % 4) less[n][i / 4] = two;
                }
            }
        }

        for (int t = run.t; t < t1; ++t) {
            if (ok) ok = warp_wait(&full[stage], phase, a.status, kSiteFull);
            if (ok) {
                const int key_tile = tiles.tile(t) * kTile;
                const uint32_t ks = smem_u32(smem) + stage * 2 * C::kHalf, vs = ks + C::kHalf;
                const int mi = lane >> 3, mr = lane & 7;
                // every key of the tile exists, and every row sees it
                const bool plain = key_tile + kTile <= tiles.len && all_seen(p_first, p_last, key_tile, key_tile + kTile - 1, a.window, a.sinks);
                float sc[C::kUnits][NT][4];  // S^T of the warp's units: keys g and g + 8, rows 2 tq and 2 tq + 1
#pragma unroll
                for (int w = 0; w < C::kUnits; ++w) {
                    const int unit = w * kWarps + warp, key0 = key_tile + unit * kUnit;
                    if constexpr (!FOUR) {
#pragma unroll
                        for (int n = 0; n < NT; ++n) sc[w][n][0] = sc[w][n][1] = sc[w][n][2] = sc[w][n][3] = 0.f;
                        const uint32_t row = kUnit * unit + mr + (mi & 1) * 8;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            uint32_t kf[4];  // 16-byte chunk c of row r of a 64-column panel sits at c ^ (r % 8)
                            const uint32_t chunk = (i & 3) * 2 + (mi >> 1);
                            ldsm4(kf, ks + (i >> 2) * (kTile * 128) + row * 128 + ((chunk ^ (row & 7)) << 4));
#pragma unroll
                            for (int n = 0; n < NT; ++n) mma16816(sc[w][n], kf, qf[n][i][0], qf[n][i][1]);
                        }
                    } else {
                        const uint32_t at = ks + unit * U::kBytes, scales = at + U::kCodes;
                        uint32_t code[2][kGroups], s2[2][kGroups / 2], by[4];
                        load_codes<D>(code, at, lane);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            load_words(s2[half], scales + 2 * U::k_scale(g + 8 * half, 0));
                            uint32_t two[1];
                            load_words(two, scales + 2 * U::k_scale(g + 8 * half, 2 * (tq % (kGroups / 2))));
                            by[half] = by[2 + half] = two[0];
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_f16_new(sc[w][n], by, less[n][0], less[n][1]);
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
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                float part[4];
                                mma_f16_new(part, x, qf[n][2 * j][0], qf[n][2 * j][1]);
                                mma_f16(part, y, qf[n][2 * j + 1][0], qf[n][2 * j + 1][1]);
                                sc[w][n][0] = fmaf(s_lo, part[0], sc[w][n][0]), sc[w][n][1] = fmaf(s_lo, part[1], sc[w][n][1]);
                                sc[w][n][2] = fmaf(s_hi, part[2], sc[w][n][2]), sc[w][n][3] = fmaf(s_hi, part[3], sc[w][n][3]);
                            }
                        }
                    }
                    if (!plain) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint32_t seen = seen_keys(position(8 * n + 2 * tq + e), key0, a.window, a.sinks);
                                if (!(seen >> g & 1u)) sc[w][n][e] = -INFINITY;
                                if (!(seen >> (g + 8) & 1u)) sc[w][n][2 + e] = -INFINITY;
                            }
                    }
                }

                // scales of the values of keys 2 tq and 2 tq + 1 (+ 8)
                uint32_t s2[FOUR ? C::kUnits : 1][2][kGroups];
                if constexpr (FOUR) {
                    uint32_t bits = 0;
#pragma unroll
                    for (int w = 0; w < C::kUnits; ++w) {
                        const int unit = w * kWarps + warp;
#pragma unroll
                        for (int half = 0; half < 2; ++half) load_words(s2[w][half], vs + unit * U::kBytes + U::kCodes + 2 * U::v_scale(2 * tq + 8 * half, 0));
                        if (!plain) {
                            // keys that no row sees: 0 times whatever their scales are must not reach O.  (A row's own keys alone
                            // where a lane holds one row: what other rows see may be no number either.)
                            const int key0 = key_tile + unit * kUnit;
                            uint32_t keep[2];
                            keep_seen(keep, NT == 1 ? seen_keys(position(g), key0, a.window, a.sinks) : used_keys(tiles, key0, a.sinks), tq);
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
                    // A weight is 2^8 at most, so its products with scales below 2^(E + 7) fit in fp16.  The scales' bits
                    // together are no less than the largest (and less than twice it, or all of 2^(1 + k) - 1 exponents).
                    const uint32_t limit = max((uint32_t)(E + 7 + 15) << 10, 0x200u);  // 2^(E + 7)
                    if (__any_sync(0xffffffffu, E < 9 && (bits + (0x8000u - limit) * 0x10001u) & 0x80008000u)) {
                        uint32_t most = 0;
#pragma unroll
                        for (int w = 0; w < C::kUnits; ++w)
#pragma unroll
                            for (int half = 0; half < 2; ++half)
#pragma unroll
                                for (int j = 0; j < kGroups; ++j) most = max_h2(most, s2[w][half][j]);
                        const float2 mh = unpack_h2(most);
                        const uint32_t all = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(mh.x, mh.y)));
                        const int need = (int)(all >> 23) - 127 - 6;
                        if (need > E) {
                            const int to = max(-6, min(9, need));
                            const float by = __int_as_float((127 + E - to) << 23), by_l = __int_as_float((127 + Ep - to) << 23);
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
#pragma unroll
                                for (int e = 0; e < 2; ++e) l[n][e] *= by_l, off[n][e] += (float)(to - Ep);
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    ones[n][e] *= by;
#pragma unroll
                                    for (int i = 0; i < D / 16; ++i) o[n][i][e] *= by;
                                }
                            }
                            E = Ep = to;
                        }
                    }
                    if (E == kTinyScales) {
#pragma unroll
                        for (int w = 0; w < C::kUnits; ++w)
#pragma unroll
                            for (int half = 0; half < 2; ++half)
#pragma unroll
                                for (int j = 0; j < kGroups; ++j) s2[w][half][j] = mul_h2(s2[w][half][j], 0x78007800u);
                    }
                }

                // the weights' logarithms; the maxima are taken again only when a weight would grow past 2^8
                bool grow = false;
                auto logs = [&](int w, int n, int e) { return fmaf(sc[w][n][e], f[n][e & 1], -off[n][e & 1]); };
                const float limit = 8.f - (FOUR ? (float)Ep : 0.f);
#pragma unroll
                for (int w = 0; w < C::kUnits; ++w)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        grow |= fmaxf(fmax3(logs(w, n, 0), logs(w, n, 1), logs(w, n, 2)), logs(w, n, 3)) > limit;
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float mt = -INFINITY;
#pragma unroll
                            for (int w = 0; w < C::kUnits; ++w) mt = fmax3(mt, sc[w][n][e], sc[w][n][2 + e]);
                            mt *= f[n][e];
                            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 4));
                            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 8));
                            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
                            mt += (float)Ep;
                            if (mt > off[n][e] + 8.f) {
                                const float alpha = ex2_approx(off[n][e] - mt);
                                l[n][e] *= alpha;
                                if constexpr (FOUR) ones[n][e] *= alpha, ones[n][2 + e] *= alpha;
#pragma unroll
                                for (int i = 0; i < D / 16; ++i) o[n][i][e] *= alpha, o[n][i][2 + e] *= alpha;
                                off[n][e] = mt;
                            }
                        }
                }

#pragma unroll
                for (int w = 0; w < C::kUnits; ++w) {
                    const int unit = w * kWarps + warp, key0 = key_tile + unit * kUnit;
                    uint32_t pb[NT][2];  // P^T as the second product's operand: row g, keys 2 tq and 2 tq + 1 (+ 8)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float p[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) p[e] = ex2_approx(logs(w, n, e));
                        // this lane's keys, not rounded; the others' are added at the end
                        l[n][0] += p[0] + p[2], l[n][1] += p[1] + p[3];
                        // the weights as operands: bf16 (half a step: up to 2^-8), or fp16 (2^-11)
                        pb[n][0] = transpose8(FOUR ? pack_h2(p[0], p[1]) : pack_bf16x2(p[0], p[1]));
                        pb[n][1] = transpose8(FOUR ? pack_h2(p[2], p[3]) : pack_bf16x2(p[2], p[3]));
                    }
                    if constexpr (!FOUR) {
                        uint32_t keep[2] = {~0u, ~0u};
                        if (!plain) keep_seen(keep, used_keys(tiles, key0, a.sinks), tq);
                        const uint32_t row = kUnit * unit + mr + (mi >> 1) * 8;
                        auto values = [&](uint32_t(&vf)[4], int i, const uint32_t(&only)[2]) {
                            const uint32_t chunk = (i & 3) * 2 + (mi & 1);
                            ldsm4t(vf, vs + (i >> 2) * (kTile * 128) + row * 128 + ((chunk ^ (row & 7)) << 4));
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
                                for (int n = 0; n < NT; ++n) mma16816(o[n][i], vf, pb[n][0], pb[n][1]);
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
                                        mma16816(sum, vf, pb[n][0], pb[n][1]);
#pragma unroll
                                        for (int e = 0; e < 4; ++e)
                                            if (position(8 * n + 2 * tq + (e & 1)) == p) o[n][i][e] = sum[e];
                                    }
                                }
                            }
                        }
                    } else {
                        uint32_t code[2][kGroups];
                        load_codes<D>(code, vs + unit * U::kBytes, lane);
                        uint32_t sees[NT][2];  // row g's own keys, where a lane holds two rows
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            sees[n][0] = sees[n][1] = ~0u;
                            if (NT > 1 && !plain) keep_seen(sees[n], seen_keys(position(8 * n + g), key0, a.window, a.sinks), tq);
                        }
#pragma unroll
                        for (int j = 0; j < kGroups; ++j) {
                            uint32_t x[4], y[4];
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                const uint32_t c = code[half][j], d = c >> 8;
                                x[2 * half] = c & 0x000f000fu, x[2 * half + 1] = c & 0x00f000f0u;
                                y[2 * half] = d & 0x000f000fu, y[2 * half + 1] = d & 0x00f000f0u;
                            }
                            const uint32_t one = g == j ? 0x3c003c00u : 0u, row_j[4] = {one, 0u, one, 0u};
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                uint32_t b0 = mul_h2(pb[n][0], s2[w][0][j]), b1 = mul_h2(pb[n][1], s2[w][1][j]);
                                if (NT > 1) b0 &= sees[n][0], b1 &= sees[n][1];
                                mma_f16(o[n][2 * j], x, b0, b1);
                                mma_f16(o[n][2 * j + 1], y, b0, b1);
                                mma_f16(ones[n], row_j, b0, b1);
                            }
                        }
                    }
                }
                warp_arrive(&empty[stage]);
            }
            if (++stage == C::kStages) stage = 0, phase ^= 1;
        }

        // Join the four warps' states, 64 channels at a time, and write them: O and L of a list that this CTA holds whole,
        // else a partial, in its first slot what began in a CTA before this one, in its second what goes on behind it.
        const bool whole = run.t == 0 && t1 == tiles.n;
        const size_t slot = ((size_t)blockIdx.x * 2 + (run.t == 0)) * kRows;
        if (run.t == 0 && !whole) {
            tail = (run.b * a.pool.Hkv + h) * a.row_tiles + run.u % a.row_tiles;
            tail_parts = 1 + (int)((tiles.n - t1 + run.count - 1) / run.count);
        }
        if (FOUR && E == kTinyScales) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    ones[FOUR ? n : 0][e] *= 0x1p-15f;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) o[n][i][e] *= 0x1p-15f;
                }
        }
        float *buf = reinterpret_cast<float *>(smem + C::kJoinOff);  // [warp][place][8 rows]
        float2 *ml = reinterpret_cast<float2 *>(smem + C::kMlOff);   // [warp][8 rows]
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 4);
                l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 8);
                l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 16);
            }
#pragma unroll
            for (int c = 0; c < D / kJoinCols; ++c) {
                asm volatile("bar.sync 1, 128;" ::: "memory");  // the buffer is free
                if (c == 0 && g < 2) ml[8 * warp + 2 * tq + g] = make_float2(l[n][g & 1] == 0.f ? -INFINITY : off[n][g & 1], l[n][g & 1]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float *to = buf + warp * (kJoinCols * 8) + 2 * tq;
                    const int i_all = 4 * c + i;
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = o[n][i_all][e];
                    int place[2] = {16 * i + g, 16 * i + g + 8};
                    if constexpr (FOUR) {
                        // channel 32 j + 4 g + (0, 1 | 2, 3) at place 8 (channel % 4) + g of its group
                        const int j = i_all / 2, k = i_all % 2;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float sum = 8.f * __shfl_sync(0xffffffffu, ones[n][e], 4 * j + tq);
                            v[e] = fmaf(v[e], 0x1p24f, -sum);
                            v[2 + e] = fmaf(v[2 + e], 0x1p20f, -sum);
                        }
                        place[0] = 32 * (j & 1) + 16 * k + g;
                        place[1] = place[0] + 8;
                    }
                    *reinterpret_cast<float2 *>(to + place[0] * 8) = make_float2(v[0], v[1]);
                    *reinterpret_cast<float2 *>(to + place[1] * 8) = make_float2(v[2], v[3]);
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
                for (int k = 0; k < kJoinCols * 8 / 2 / (32 * kWarps); ++k) {
                    const int r = threadIdx.x & 7, ch = 2 * ((threadIdx.x >> 3) + 16 * k);  // a row, a pair of channels
                    const int at = FOUR ? 32 * (ch / 32) + 8 * (ch % 4) + ch % 32 / 4 : ch, next = at + (FOUR ? 8 : 1);
                    float M = -INFINITY, ls = 0.f;
                    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[8 * w + r].x);
                    const float Mb = M == -INFINITY ? 0.f : M;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float fw = ex2_approx(ml[8 * w + r].x - Mb);
                        ls = fmaf(ml[8 * w + r].y, fw, ls);
                        acc.x = fmaf(buf[w * (kJoinCols * 8) + at * 8 + r], fw, acc.x);
                        acc.y = fmaf(buf[w * (kJoinCols * 8) + next * 8 + r], fw, acc.y);
                    }
                    const int row = 8 * n + r, col = kJoinCols * c + ch;
                    if (row0 + row >= a.R) continue;
                    if (whole) {
                        const float inv = ls > 0.f ? 1.f / ls : ls == 0.f ? 0.f : ls;
                        reinterpret_cast<uint32_t *>(a.o)[((first_row + row) * D + col) / 2] = pack_bf16x2(acc.x * inv, acc.y * inv);
                        if (col == 0) a.lse[first_row + row] = (M + __log2f(ls)) * 0.69314718055994531f;
                    } else {
                        *reinterpret_cast<float2 *>(a.part_o + (slot + row) * D + col) = acc;
                        if (col == 0) a.part_ml[slot + row] = make_float2(M, ls);
                    }
                }
            }
        }
        left -= t1 - run.t;
        run.t = 0;
        if (++run.u == per_seq) run.u = 0, ++run.b;
    }
    if (a.tails && threadIdx.x == 0) a.tails[blockIdx.x] = make_int2(tail, tail_parts);
}

// Adds up the partials of the list that goes on behind CTA blockIdx.x of the kernel before, if one does: the CTA's second
// slot and the first ones of the CTAs behind it.  One row a CTA; a thread owns four columns of every kWays-th partial.
template <int D>
__global__ void __launch_bounds__(128) paged_join_kernel(PagedDecodeArgs a, int rows) {
    constexpr int kCols = D / 4, kWays = 128 / kCols;
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

template <int D, int NT, bool FOUR>
cudaError_t launch_d(const PagedDecodeArgs &a, int ctas, const CUtensorMap &tk, const CUtensorMap &tv, cudaStream_t s) {
    using C = Cfg<D, NT, FOUR>;
    auto kern = paged_decode_kernel<D, NT, FOUR>;
    static std::atomic<unsigned long long> allowed{0};
    cudaError_t e = allow_smem((const void *)kern, C::kAlloc, allowed);
    if (e == cudaSuccess) e = launch_behind(kern, dim3(ctas), kThreads, C::kAlloc, false, 1, s, tk, tv, a);
    if (e == cudaSuccess && a.tails) e = launch_behind(paged_join_kernel<D>, dim3(ctas, std::min(a.R, 8 * NT)), 128, 0, true, 1, s, a, 8 * NT);
    return e;
}

template <int D, int NT, bool FOUR>
PagedPlan plan_d() {
    using C = Cfg<D, NT, FOUR>;
    return PagedPlan{C::kTile, 8 * NT, C::kCtas};
}

// 8 rows a CTA, or 16 where there are more: twice the products for half the reads.  (4-bit heads of 256: 8; with 16 the
// accumulators alone would take a thread's registers.)
bool sixteen(int R, int D, bool four) { return R > 8 && !(four && D == 256); }

}  // namespace

PagedPlan paged_plan(int R, int D, bool four) {
    const bool two = sixteen(R, D, four);
    switch (D) {
        case 64: return four ? (two ? plan_d<64, 2, true>() : plan_d<64, 1, true>()) : two ? plan_d<64, 2, false>() : plan_d<64, 1, false>();
        case 128: return four ? (two ? plan_d<128, 2, true>() : plan_d<128, 1, true>()) : two ? plan_d<128, 2, false>() : plan_d<128, 1, false>();
        default: return four ? plan_d<256, 1, true>() : two ? plan_d<256, 2, false>() : plan_d<256, 1, false>();
    }
}

cudaError_t launch_paged_decode(const PagedDecodeArgs &a, bool four, int ctas, const CUtensorMap &tk, const CUtensorMap &tv, cudaStream_t s) {
    const bool two = sixteen(a.R, a.D, four);
    switch (a.D) {
        case 64:
            return four ? (two ? launch_d<64, 2, true>(a, ctas, tk, tv, s) : launch_d<64, 1, true>(a, ctas, tk, tv, s))
                        : two ? launch_d<64, 2, false>(a, ctas, tk, tv, s) : launch_d<64, 1, false>(a, ctas, tk, tv, s);
        case 128:
            return four ? (two ? launch_d<128, 2, true>(a, ctas, tk, tv, s) : launch_d<128, 1, true>(a, ctas, tk, tv, s))
                        : two ? launch_d<128, 2, false>(a, ctas, tk, tv, s) : launch_d<128, 1, false>(a, ctas, tk, tv, s);
        case 256:
            return four ? launch_d<256, 1, true>(a, ctas, tk, tv, s)
                        : two ? launch_d<256, 2, false>(a, ctas, tk, tv, s) : launch_d<256, 1, false>(a, ctas, tk, tv, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace fa
