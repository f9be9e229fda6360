// win.cuh -- windowed attention: which keys a tile of query rows reads, and
// which of them each row sees.
//
// Row i of N_q query rows sits at position p = i + N_k - N_q and sees key j iff
//   j <= p  and  (j < sinks  or  j > p - window):
// the `window` last keys up to its own and the first `sinks` keys.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace fa {

// The longest key range windowed attention takes: sums and differences of two positions and a window
// then stay inside 32 bits.
constexpr int kMaxPositions = 1 << 29;

// The most products that one accumulator adds up.  The tensor cores align a sum's addends and drop what lies 2^-25 and
// more below it, so n products of one sign and about the same size lose n 2^-27 of their sum, up to n 2^-26 (measured, O of
// one row and dV of one key: 0.8 % at 2^20, 1.4 % at 2^21, 5 % at 2^23; at 2^25 the sum stops growing).  Up to here
// that is within the 2e-2 that the bf16 results are held to.
constexpr int kMaxSum = 1 << 21;

// The key tiles (bn keys each) that positions p0 .. p1 read: n_sink tiles from key 0 on, then tiles from
// key lo on, n in all.  A window tile starts at the first key that p0 sees rather than at a multiple of
// bn, so a tile of 128 rows reads window + 127 keys and not up to bn - 1 more.  Where the window reaches the
// sinks there is one range from key 0 (n_sink = 0); otherwise the sink tiles stand for the sinks alone (their
// window is 0: a key that a sink tile and a window tile both hold counts in the window tile), so every key that
// the tiles stand for is seen by one of the positions or by a later one.
struct KeySpan {
    int n_sink, lo, n;
    __host__ __device__ int key0(int j, int bn) const { return j < n_sink ? j * bn : lo + (j - n_sink) * bn; }
    __host__ __device__ int window_in(int j, int window) const { return j < n_sink ? 0 : window; }
};

__host__ __device__ inline KeySpan key_span(int p0, int p1, int window, int sinks, int bn) {
    KeySpan s;
    const int lo = p0 - window + 1;
    const bool gap = lo > sinks;
    s.n_sink = gap ? (sinks + bn - 1) / bn : 0;
    s.lo = gap ? lo : 0;
    s.n = s.n_sink + (p1 + 1 - s.lo + bn - 1) / bn;
    return s;
}

// bits [0, n) of a word
__host__ __device__ inline uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// bit i: position p sees key k0 + i (i < 32)
__host__ __device__ inline uint32_t seen_keys(int p, int k0, int window, int sinks) {
    return low_bits(p + 1 - k0) & (~low_bits(p - window + 1 - k0) | low_bits(sinks - k0));
}

// every one of positions p0 .. p1 sees every one of keys k0 .. k1
__host__ __device__ inline bool all_seen(int p0, int p1, int k0, int k1, int window, int sinks) {
    return k1 <= p0 && (k0 > p1 - window || k1 < sinks);
}

// bit i: the position p0 + i sees key (i < 32)
__host__ __device__ inline uint32_t seeing_positions(int key, int p0, int window, int sinks) {
    return ~low_bits(key - p0) & (key < sinks ? ~0u : low_bits(key + window - p0));
}

// Windowed (and grouped-head) form of the backward kernels' arguments; unused by their plain forms.
struct WinArgs {
    int Hkv;     // key heads; query head h reads key head h / (H / Hkv)
    int Nk;      // keys; the query rows are the last N of the Nk positions
    int window, sinks;
    // dK/dV: rows far behind the sinks see the sinks alone, and one CTA per sink tile would walk all of them.
    // They are cut into `chunks` work items per sink tile (0: not cut); those items and the sink tile's own
    // write fp32 partials, which sink_sum_kernel adds in a fixed order.
    int sink_tiles, chunks;
    int few;  // the chunks run in win_sinks.cu instead (one sink tile of at most kFewSinks sinks, D = 64)
};
constexpr int kFewSinks = 16;
// Rows at positions below this have their D_i from win_delta.cu.
constexpr int kExactDelta = 128;

// Division of 0 <= n < 2^31 by a number that the host knows, by a multiplication (Granlund and Montgomery, "Division by
// invariant integers using multiplication", 1994): n / d = (mulhi(n, mul) + n) >> shift.
struct FastDiv {
    uint32_t d, mul, shift;
    FastDiv() = default;
    explicit FastDiv(uint32_t by) : d(by), mul(0), shift(0) {
        while ((1ull << shift) < by) ++shift;
        mul = (uint32_t)(((1ull << 32) * ((1ull << shift) - by)) / by + 1);
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int div(int n) const {
        return (int)((__umulhi((uint32_t)n, mul) + (uint32_t)n) >> shift);
    }
#endif
};

// Partials of the shared prefix: unnormalised O, m (log2 units) and l of every packed 128-row query tile and chunk of
// the prefix.  O lies in groups of 8 columns, [key head][tile][chunk][D / 8][128 rows][8], so that the 32 rows of a warp
// write one contiguous KB per instruction (rows of D floats each: 3900 cycles a tile instead of 1100).
struct PrefixParts {
    float *o;                 // 32-byte aligned
    float2 *ml;               // [key head][tile][chunk][128 rows]
    int m_tiles, splits;
    int R, rb, nb;            // rows of a (sequence, key head); a tile holds rb rows of each of nb sequences
#ifdef __CUDACC__
    // first of the tile's chunks in units of 128-row partials
    __device__ __forceinline__ size_t at(int h, int tile) const { return ((size_t)h * m_tiles + tile) * splits; }
    // the tile of row rr of sequence b, and the row's place in it
    __device__ __forceinline__ void place(int b, int rr, int *tile, int *r) const {
        if (R <= rb) {
            *tile = b / nb;
            *r = b % nb * rb + rr;
        } else {
            *tile = b * ((R + rb - 1) / rb) + rr / rb;
            *r = rr % rb;
        }
    }
#endif
};

// The forward over the keys that a span of query rows sees (win_fwd.cu, and fwd_bf16.cu for wide heads).
// Two forms: windowed attention writes O and LSE; the shared-prefix form packs the rows of all sequences
// into 128-row tiles, sees every key, and writes the partials above.
struct SpanArgs {
    void *o;
    float *lse;
    int B, Hq, Hkv, Nq, Nk, D;
    int window, sinks;
    float scale_log2;
    int *status;
    int num_sms;
    // windowed: query heads of all sequences, of one, of a key head
    FastDiv per_rows, per_seq, group;
    // shared prefix (parts.o set): chunks of chunk_tiles key tiles
    PrefixParts parts;
    int chunk_tiles;
};
// Keys of the K/V tiles of the windowed forward at head dimension D.
inline int win_fwd_keys(int D) { return D <= 64 ? 128 : 64; }

cudaError_t launch_win_fwd(const SpanArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                           const CUtensorMap &tks, const CUtensorMap &tvs, const CUtensorMap &to, cudaStream_t s);
cudaError_t launch_win_fwd_wide(const SpanArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                                const CUtensorMap &tks, const CUtensorMap &tvs, cudaStream_t s);

}  // namespace fa
