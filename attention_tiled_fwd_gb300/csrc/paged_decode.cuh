// paged_decode.cuh -- what the decode kernels over bf16 and over 4-bit pages share: the list of tiles, its cut into runs, and
// the join of the warps' states.
#pragma once
#include "paged.cuh"
#include "sm100_ptx.cuh"

namespace fa {

constexpr int kDecodeWarps = 4;  // warps that compute
constexpr int kJoinCols = 64;    // channels that they join at a time
constexpr float kNone = -3e38f;  // the running maximum of a row that has seen nothing

// Waits as in sm100_ptx.cuh, by a whole warp, in steps of up to 1 ms that the hardware sleeps through: the polls of warps that
// wait would take issue slots from those that compute.
__device__ __forceinline__ bool sleepy_try(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(1000000u)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ bool sleepy_wait(uint64_t *bar, uint32_t parity, int *status, int site) {
    const uint32_t b = smem_u32(bar);
    if (__all_sync(0xffffffffu, sleepy_try(b, parity))) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        if (__all_sync(0xffffffffu, sleepy_try(b, parity))) return true;
        if (__any_sync(0xffffffffu, globaltimer_ns() - t0 > kWaitLimitNs)) break;
    }
    if ((threadIdx.x & 31) == 0) record_failure(status, 8 /* FA_ERR_TIMEOUT */, site);
    return false;
}

// The 8 x 8 matrix of 16-bit values that the warp holds, a row in four lanes, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
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

// This CTA's run: `count` steps from step v of list u of sequence b on.  A list of n tiles has COST steps for what it costs
// besides (q, the join, the stores: about that many tiles' time), and then a step for each tile.
template <int COST>
struct Run {
    int b, u, v;
    long long count;
    // Tiles [t0, t1) of the present list of n, of `left` steps.
    __device__ __forceinline__ void part(int n, long long left, int *t0, int *t1) const {
        *t0 = max(0, v - COST);
        *t1 = max(0, (int)min((long long)(n + COST), v + left) - COST);
    }
    // On to the next list; the steps that are left then.
    __device__ __forceinline__ long long next(int n, long long left, int lists) {
        left -= n + COST - v;
        v = 0;
        if (++u == lists) u = 0, ++b;
        return left;
    }
};

constexpr int kScan = 80;    // bytes of shared memory that finding the run takes, and its result stays in
constexpr int kAllOff = 72;  // of them, the number of all steps

// CTAs that hold a part of the list that goes on `rest` steps behind this CTA's run, this one among them.
static __device__ __noinline__ int parts_behind(const WorkCut &cut, long long all, int rest) {
    const long long end = cut.begin(blockIdx.x + 1, all) + rest;
    int c = 2;
    while (cut.begin(blockIdx.x + c, all) < end) ++c;
    return c;
}

// All threads: each adds up the steps of its share of the sequences, and the one whose share the run begins in finds where.
template <int TILE, int THREADS, int COST>
__device__ __forceinline__ Run<COST> find_run(const PagedDecodeArgs &a, uint8_t *scratch) {
    long long *totals = reinterpret_cast<long long *>(scratch);
    int *where = reinterpret_cast<int *>(scratch + 8 * (THREADS / 32));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = (a.B + THREADS - 1) / THREADS, b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += Tiles::of<TILE>(a, b).n + COST;
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
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += totals[w];
        total += totals[w];
    }
    const long long lists = (long long)a.pool.Hkv * a.row_tiles, all = total * lists;
    const long long begin = a.cut.begin(blockIdx.x, all);
    Run<COST> r;
    r.count = a.cut.begin(blockIdx.x + 1, all) - begin;
    if (threadIdx.x == 0) *reinterpret_cast<long long *>(scratch + kAllOff) = all;  // for parts_behind
    if (begin >= before * lists && begin < (before + mine) * lists) {
        for (int b = b0;; ++b) {
            const int n = Tiles::of<TILE>(a, b).n + COST;
            if (begin < (before + n) * lists) {
                const long long in = begin - before * lists;
                where[0] = b;
                where[1] = in >> 31 ? (int)(in / n) : (int)((unsigned)in / (unsigned)n);  // (64 bits take longer)
                where[2] = (int)(in - (long long)where[1] * n);
                break;
            }
            before += n;
        }
    }
    __syncthreads();
    r.b = r.u = r.v = 0;
    if (r.count > 0) r.b = where[0], r.u = where[1], r.v = where[2];
    return r;
}

// The four warps' states of 8 rows, joined: ml [warp][8 rows] their maxima and sums.  Row threadIdx.x % 8: the factors of the
// warps' sums, the joined maximum and sum.
struct JoinedRow {
    float f[kDecodeWarps], M, l;
    __device__ __forceinline__ void read(const float2 *ml) {
        const float2 *row = ml + (threadIdx.x & 7);
        M = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < kDecodeWarps; ++w) M = fmaxf(M, row[8 * w].x);
        const float Mb = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int w = 0; w < kDecodeWarps; ++w) {
            f[w] = ex2_approx(row[8 * w].x - Mb);
            l = fmaf(row[8 * w].y, f[w], l);
        }
    }
};

// buf [warp][64 places][8 rows]: 64 channels of the warps' sums, channel 2 i of a pair at place `at(2 i)` and 2 i + 1 `next` places
// behind it.  Written as O and L of the rows that exist where the CTA holds the whole list (`whole`), else to the partial `slot`.
// 128 threads.
template <int D, int NEXT, class At>
__device__ __forceinline__ void join_warps(const PagedDecodeArgs &a, float *part_o, float2 *part_ml, const float *buf, const JoinedRow &j,
                                           bool whole, size_t slot, size_t first_row, int row8, int rows, int col0, At at) {
    const int r = threadIdx.x & 7, row = row8 + r;
    if (row >= rows) return;
    const float inv = !whole ? 1.f : j.l > 0.f ? 1.f / j.l : j.l == 0.f ? 0.f : j.l;
#pragma unroll
    for (int k = 0; k < kJoinCols * 8 / 2 / 128; ++k) {
        const int ch = 2 * ((threadIdx.x >> 3) + 16 * k), place = at(ch), col = col0 + ch;  // a pair of channels
        float2 acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kDecodeWarps; ++w) {
            acc.x = fmaf(buf[w * (kJoinCols * 8) + place * 8 + r], j.f[w], acc.x);
            acc.y = fmaf(buf[w * (kJoinCols * 8) + (place + NEXT) * 8 + r], j.f[w], acc.y);
        }
        if (whole) {
            reinterpret_cast<uint32_t *>(a.o)[((first_row + row) * D + col) / 2] = pack_bf16x2(acc.x * inv, acc.y * inv);
            if (col == 0) a.lse[first_row + row] = (j.M + __log2f(j.l)) * 0.69314718055994531f;
        } else {
            *reinterpret_cast<float2 *>(part_o + (slot + row) * D + col) = acc;
            if (col == 0) part_ml[slot + row] = make_float2(j.M, j.l);
        }
    }
}

// A CTA's share of a list whose CTAs are a cluster.
template <int TILE, int COST>
__device__ __forceinline__ Run<COST> cluster_run(const PagedDecodeArgs &a, uint8_t *scratch) {
    const int list = blockIdx.x / a.cluster, rank = blockIdx.x - list * a.cluster, per_seq = a.pool.Hkv * a.row_tiles;
    Run<COST> r;
    r.b = list / per_seq;
    r.u = list - r.b * per_seq;
    const int n = Tiles::of<TILE>(a, r.b).n, t0 = n * rank / a.cluster;
    r.v = t0 + COST;
    r.count = n * (rank + 1) / a.cluster - t0;
    if (threadIdx.x == 0) *reinterpret_cast<int *>(scratch) = n;  // for join_cluster
    __syncthreads();
    return r;
}

// The partials of a cluster's list (each in its CTA's shared memory, the same place in all), joined by all of the CTAs, a share
// of the rows' columns each.  128 threads.
template <int D>
__device__ __noinline__ void join_cluster(const PagedDecodeArgs &a, const float *part_o, const float2 *part_ml, int n, int tile_rows) {
    const int list = blockIdx.x / a.cluster, rank = blockIdx.x - list * a.cluster;
    const int row0 = list % a.row_tiles * tile_rows, rows = min(tile_rows, a.R - row0);
    const size_t first_row = (size_t)(list / a.row_tiles) * a.R + row0;
    const uint32_t at_o = smem_u32(part_o), at_ml = smem_u32(part_ml);
    cluster_sync();
    for (int idx = rank * 128 + threadIdx.x; idx < rows * (D / 4); idx += a.cluster * 128) {
        const int r = idx / (D / 4), c = idx % (D / 4) * 4;
        float M = -INFINITY, l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kBatch = 8;
        for (int s0 = 0; s0 < a.cluster; s0 += kBatch) {
            float2 ml[kBatch];
            float4 v[kBatch];
            float Mn = M;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int s = s0 + i;
                ml[i] = make_float2(-INFINITY, 0.f);
                v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (s >= a.cluster || n * s / a.cluster == n * (s + 1) / a.cluster) continue;  // (no share: nothing written)
                ml[i] = ld_cluster_f2(map_to_cta(at_ml + r * 8, s));
                v[i] = ld_cluster_f4(map_to_cta(at_o + (r * D + c) * 4, s));
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) Mn = fmaxf(Mn, ml[i].x);
            const float Mb = Mn == -INFINITY ? 0.f : Mn, f0 = ex2_approx(M - Mb);
            l *= f0;
            acc.x *= f0, acc.y *= f0, acc.z *= f0, acc.w *= f0;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const float f = ex2_approx(ml[i].x - Mb);
                l = fmaf(ml[i].y, f, l);
                acc.x = fmaf(v[i].x, f, acc.x);
                acc.y = fmaf(v[i].y, f, acc.y);
                acc.z = fmaf(v[i].z, f, acc.z);
                acc.w = fmaf(v[i].w, f, acc.w);
            }
            M = Mn;
        }
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
        const size_t row = first_row + r;
        uint2 w;
        w.x = pack_bf16x2(acc.x * inv, acc.y * inv);
        w.y = pack_bf16x2(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + row * D + c) = w;
        if (c == 0) a.lse[row] = (M + __log2f(l)) * 0.69314718055994531f;
    }
    cluster_sync();  // no CTA leaves while another reads its partial
}

__device__ __forceinline__ void sync_warps() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

}  // namespace fa
