// paged.cuh -- a cache of keys and values in pages, and where its 4-bit form holds what.
//
// A pool holds n_pages pages of `page` positions (a power of two, 16 or more) for every key head; sequence b's position p
// is row p % page of page table[b][p / page].  bf16 pages are [n_pages, Hkv, page, D].  4-bit pages are bytes
// [n_pages, Hkv, page, 9 D / 16], of which every 16 positions are a unit of 9 D bytes: 8 D of codes, D of scales.  A value
// is scale (code - 8), code in 1 .. 15, with one fp16 scale for 32 channels of one position (4.5 bits a value).
//
// The order inside a unit is that of the tensor cores' fragments, so that the decode kernel reads its operands from shared
// memory 16 bytes a lane, with no conflict and nothing to rearrange.  Codes are 32-bit words, word(half, group, lane):
//   keys    half = position / 8, lane = 4 (position % 8) + (channel % 32) / 8: 8 channels of a position
//   values  half = position / 8, lane = 4 ((channel % 32) / 4) + (position % 8) / 2: 4 channels of an even position in the
//           low half, of the odd position behind it in the high half (a position never shares a byte with another)
// the lowest channel in the lowest bits.  Scales: keys [position][group], values [position / 2][group][position % 2].
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include "win.cuh"

namespace fa {

constexpr int kUnit = 16;                // positions of a unit of 4-bit pages, and the least page
constexpr int kMaxPage = 256;
constexpr int kMaxCapacity = 1 << 23;    // positions of a sequence: sums of 2^21 keys a warp are tested, longer ones are not
constexpr int kErrPage = 13;             // FA_ERR_PAGE in the status word

template <int D>
struct Unit4 {
    static constexpr int kGroups = D / 32;
    static constexpr int kWide = kGroups < 4 ? kGroups : 4;  // neighbouring words of a lane: its groups, 16 bytes at most
    static constexpr int kCodes = 8 * D, kBytes = 9 * D;
    static __host__ __device__ constexpr int word(int half, int group, int lane) {
        return ((half * (kGroups / kWide) + group / kWide) * 32 + lane) * kWide + group % kWide;
    }
    // scales, counted in fp16
    static __host__ __device__ constexpr int k_scale(int pos, int group) { return pos * kGroups + group; }
    static __host__ __device__ constexpr int v_scale(int pos, int group) { return ((pos >> 1) * kGroups + group) * 2 + (pos & 1); }
};

// bytes of `rows` positions of a page and head
inline __host__ __device__ long long page_row_bytes(int D, bool four) { return four ? 9 * D / 16 : 2 * D; }

struct PagePool {
    uint8_t *k, *v;
    const int *table;  // [B][slots]
    int n_pages, shift, slots, Hkv;
    __host__ __device__ int capacity() const { return slots << shift; }
#ifdef __CUDACC__
    // The table's entry for position p of sequence b.
    __device__ __forceinline__ int entry(int b, int p) const { return __ldg(table + (size_t)b * slots + (p >> shift)); }
    // The page that holds it, or -1 where the table has none of the pool's there.
    __device__ __forceinline__ int page_of(int b, int p) const {
        const int at = entry(b, p);
        return (unsigned)at < (unsigned)n_pages ? at : -1;
    }
    // First byte of row p % page of a page and head, rows of `bytes` bytes (4-bit pages: p a multiple of 16).
    __device__ __forceinline__ size_t at(int page, int h, int p, int bytes) const {
        return ((((size_t)page * Hkv + h) << shift) + (p & ((1 << shift) - 1))) * bytes;
    }
#endif
};

// Rows entering the cache (paged_cache.cu).  Row i of the n of sequence b sits at position lens[b] - n + i; the last
// counts[b] of them are new.
struct AppendArgs {
    const void *q, *k, *v;             // bf16 rows of D; q may be null
    long long sq[3], sk[3], sv[3];     // strides in elements: sequence, head, row
    const float *cos, *sin;            // [positions][rot / 2]
    const int *lens, *counts;
    void *q_out;                       // [B, Hq, n, D]
    PagePool pool;
    int B, Hq, n, D, rot, interleaved;
    int *status;
};
cudaError_t launch_paged_append(const AppendArgs &a, bool four, cudaStream_t s);

// The sequences' rows, contiguous: k, v [B, Hkv, rows, D] bf16, of which the first min(lens[b], rows) are written.
struct GatherArgs {
    PagePool pool;
    const int *lens;
    void *k, *v;
    int B, rows, D;
    int *status;
};
cudaError_t launch_paged_gather(const GatherArgs &a, bool four, cudaStream_t s);

// The cut of a list of work into equal runs for the CTAs of a grid, `step` of 2^64 each.  A little work is cut into whole equal runs
// instead, so that no CTA between two that work has none.
struct WorkCut {
    unsigned long long step;
#ifdef __CUDACC__
    __device__ __forceinline__ long long begin(unsigned cta, long long total) const {
        if (cta >= gridDim.x) return total;
        if (total < 16ll * gridDim.x) return min(total, (long long)(((unsigned)total + gridDim.x - 1) / gridDim.x) * cta);
        return (long long)__umul64hi((unsigned long long)total, cta * step);
    }
#endif
};

struct PagedDecodeArgs {
    const void *q;     // [B, Hkv, R, D] bf16, R = (Hq / Hkv) n_q: the caller's [B, Hq, n_q, D]
    const int *lens;   // [B], clamped to [0, capacity]; null: capacity
    void *o;           // [B, Hkv, R, D] bf16
    float *lse;        // [B, Hkv, R]
    PagePool pool;
    int B, R, n_q, D;
    int window, sinks;
    float scale_log2;
    int *status;
    int row_tiles;     // CTAs that share a key head's rows
    int cluster;       // 0: the work is cut into runs; else the CTAs of a cluster share a list and join its partials
    WorkCut cut;
    // two partials a CTA, [2 CTA + slot][rows of a tile]: O, (m, l); and the list that goes on behind a CTA (its number and
    // its partials, -1: none).  All null where no list can be cut.
    float *part_o;
    float2 *part_ml;
    int2 *tails;
};
// Keys of a tile, rows of a row tile, CTAs an SM holds, and the most tiles for a CTA of a cluster, for a decode of R rows a key head.
struct PagedPlan {
    int tile, rows, per_sm, per_cluster;
};
PagedPlan paged_plan(int R, int D, int page);  // bf16 pages
PagedPlan paged_plan4(int D);                  // 4-bit pages
// tk, tv: the pools' tensor maps (boxes of 64 columns and of the rows of a page, at most a tile's).
cudaError_t launch_paged_decode(const PagedDecodeArgs &a, int ctas, const CUtensorMap &tk, const CUtensorMap &tv, cudaStream_t s);
cudaError_t launch_paged_decode4(const PagedDecodeArgs &a, int ctas, cudaStream_t s);
// Behind either, where a list can be cut: rows of a row tile.
cudaError_t launch_paged_join(const PagedDecodeArgs &a, int ctas, int rows, cudaStream_t s);

}  // namespace fa
