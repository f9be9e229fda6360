// fa_internal.h -- launch interfaces shared by the C-ABI layer (fa_api.cu) and
// the kernel translation units.  Not part of the public ABI.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "win.cuh"

namespace fa {

// Spec table of the bf16 forward: query rows per CTA, keys per K/V tile, K/V
// ring depth, keyed by head dimension.  Picked so that the score, P and O
// buffers fit the 512 TMEM columns and the staged tiles fill (but do not
// exceed) shared memory.
//   D = 64, 128: two 128-row query tiles per CTA (fwd_bf16_pair.cu), causal
//                and non-causal, on a persistent grid of one CTA per SM; TMEM
//                per tile S 128 (P over its first 64) + O D columns; shared
//                memory 2 Q tiles + ring.
//   D = 192, 256: one 128-row query tile, two softmax warpgroups splitting
//                the columns (fwd_bf16.cu); TMEM S 2x64 + P 2x32 + O D (one
//                N = D accumulator, D-blocked shared-memory panels).
struct FwdSpec {
    int D, BM, BN, nslot;
};
constexpr FwdSpec kFwdSpecs[] = {
    {64, 256, 128, 4},   // Q 2 x 16 KB + 4 x 16 KB ring (6, 8, 10 slots measured 0-5 % slower; 5, 7, 9 more)
    {128, 256, 128, 4},  // Q 2 x 32 KB + 4 x 32 KB ring + 32 KB staging for O's TMA stores
    {192, 128, 64, 7},   // Q 48 KB + 7 x 24 KB ring (4, 5 slots measured 4-13 % slower)
    {256, 128, 64, 4},   // Q 64 KB + 4 x 32 KB ring (3 slots measured 19 % slower)
};

// Tile rows of the backward kernels' streamed operands (TMA box heights).
constexpr int kDqKRows = 64;    // dQ kernel: 128 query rows per CTA, 64-key K/V tiles
constexpr int kDkdvQRows = 64;  // dK/dV kernel: 128 keys per CTA, 64-query Q/dO tiles

// Work order of a 1-D grid over (tile, batch*head).  Causal launches go by
// tile rank, rank 0 (the most K/V tiles) first, so that the hardware, which
// dispatches CTAs in index order, starts every SM on the longest tiles and
// fills the tail with short ones.  The ranks run across groups of `group`
// heads, one group after the other, so that the K/V (or Q/dO) tiles that a
// group's CTAs stream stay in L2 between the CTAs that read them; a group of
// every head is the plain rank order.  Non-causal tiles are equal, so the
// tiles of one head stay adjacent (they share its K/V in L2).
#ifdef __CUDACC__
__device__ __forceinline__ void tile_order_at(int L, int n_tiles, int n_bh, bool causal, int group, int *rank,
                                              int *bh) {
    if (causal && (group < 1 || group >= n_bh)) {
        *rank = L / n_bh;
        *bh = L % n_bh;
    } else if (causal) {
        const int g = group;
        const int per = n_tiles * g;        // items of a full group
        const int gi = L / per;             // L's group
        const int g0 = gi * g;              // its first head
        const int gs = min(g, n_bh - g0);   // its heads (the last group may have fewer)
        const int in = L - gi * per;
        *rank = in / gs;
        *bh = g0 + in % gs;
    } else {
        *rank = L % n_tiles;
        *bh = L / n_tiles;
    }
}

__device__ __forceinline__ void tile_order(int n_tiles, int n_bh, bool causal, int group, int *rank, int *bh) {
    tile_order_at(blockIdx.x, n_tiles, n_bh, causal, group, rank, bh);
}

// The k-th work item of CTA c in a persistent grid of G CTAs (one per SM): round k of the 1-D work
// order above is dealt out forwards in even rounds and backwards in odd ones, so a CTA that drew a heavy
// item in one round draws a light one in the next.  -1: no item for this CTA in round k.
__device__ __forceinline__ int persistent_work_index(int k, int n_work) {
    const int G = gridDim.x, c = blockIdx.x;
    const int Lw = k * G + ((k & 1) ? G - 1 - c : c);
    return Lw < n_work ? Lw : -1;
}
#endif

struct FwdArgs {
    const void *q, *k, *v;
    void *o;
    float *lse;
    int B, H, N, D;
    float scale;       // softmax scale
    float scale_log2;  // scale * log2(e): scores go straight to the base-2 domain
    int causal;
    int *status;       // device status word (bounded-wait failures)
    int num_sms;       // SMs of the device: the persistent forward runs one CTA per SM
    int head_group;    // heads per group of the causal work order (tile_order_at)
    // The persistent forwards' work counter (two ints, zero between launches: the next item to draw and
    // the CTAs that have stopped drawing; the last of them zeroes both).  Null: the static deal
    // persistent_work_index, used when the whole launch's K/V fits in L2.
    int *work;
};

struct BwdArgs {
    const void *q, *k, *v, *o, *dO;
    const float *lse;
    float *delta;        // written by the dQ kernel, read by the dK/dV kernel
    void *dq, *dk, *dv;  // grad_dtype
    int B, H, N, D;
    float scale, scale_log2;
    int causal;
    int grad_bf16;  // 1: gradients stored as bf16, 0: fp32
    int *status;
    int head_group;  // heads per group of the causal work order (tile_order_at)
    WinArgs win;     // windowed kernels (WIN = true) only; N is then the query rows
};

#ifdef __CUDACC__
// Query tile x (bm rows) of the windowed dQ kernels and its key tiles (bn keys), in longest-first order: the last rows of
// every head first.
struct WinRowItem {
    int bh, kv_bh, row0, pos0;
    KeySpan span;
};

__device__ __forceinline__ WinRowItem win_row_item(const BwdArgs &a, int x, int bm, int bn) {
    const int n_bh = a.B * a.H;
    WinRowItem w;
    w.bh = x % n_bh;
    w.row0 = ((a.N + bm - 1) / bm - 1 - x / n_bh) * bm;
    w.kv_bh = w.bh / a.H * a.win.Hkv + w.bh % a.H / (a.H / a.win.Hkv);
    w.pos0 = a.win.Nk - a.N + w.row0;
    w.span = key_span(w.pos0, min(a.win.Nk, w.pos0 + bm) - 1, a.win.window, a.win.sinks, bn);
    return w;
}

// The query rows of windowed attention that keys k0 .. k0 + bk - 1 meet: rows from `first` on in `per_head`
// tiles of bq rows, for each of the key head's query heads.
struct WinRows {
    int first, per_head;
    __device__ __forceinline__ int row0(int i, int bq) const { return first + i % per_head * bq; }
};

// A work item of the windowed dK/dV kernels: tiles i0 .. i0 + n - 1 of `rows` against one key tile.  part < 0: the
// item owns its key tile's gradients; else it writes partial `part`.
struct WinKeyItem {
    int k_tile, bh, part, i0, n;
    WinRows rows;
};

__device__ __forceinline__ WinKeyItem win_key_item(const BwdArgs &a, int x, int bk, int bq) {
    const int G = a.H / a.win.Hkv, n_bh = a.B * a.win.Hkv;
    const int off = a.win.Nk - a.N;  // position of row 0
    const int extra = n_bh * a.win.sink_tiles * a.win.chunks;  // the chunks come first
    WinKeyItem w;
    int chunk = -1;
    if (x < extra) {
        chunk = x % a.win.chunks;
        w.k_tile = x / a.win.chunks % a.win.sink_tiles;
        w.bh = x / (a.win.chunks * a.win.sink_tiles);
    } else {
        w.k_tile = (x - extra) / n_bh;
        w.bh = (x - extra) % n_bh;
    }
    const int k0 = w.k_tile * bk;
    const bool cut = a.win.chunks > 0 && w.k_tile < a.win.sink_tiles;
    w.part = cut ? (w.bh * a.win.sink_tiles + w.k_tile) * (1 + a.win.chunks) + 1 + chunk : -1;
    w.rows.first = max(0, k0 - off);
    // every later row for a sink tile that is not cut, else the rows whose window holds one of the keys
    const int end = k0 < a.win.sinks && !cut ? a.N : min(a.N, k0 + bk - 1 + a.win.window - off);
    w.rows.per_head = end > w.rows.first ? (end - w.rows.first + bq - 1) / bq : 0;
    if (chunk >= 0) {  // the rows behind those
        w.rows.first += w.rows.per_head * bq;
        w.rows.per_head = a.N > w.rows.first ? (a.N - w.rows.first + bq - 1) / bq : 0;
    }
    w.i0 = 0;
    w.n = w.rows.per_head * G;
    if (chunk >= 0) {
        const int per = (w.n + a.win.chunks - 1) / a.win.chunks;
        w.i0 = min(w.n, chunk * per);
        w.n = min(w.n - w.i0, per);
    }
    return w;
}

// Walks an item's tiles without a division per tile: row of the tile, and its query slice (batch and head).
struct WinRowWalk {
    int h, slice, per_head;
    __device__ __forceinline__ WinRowWalk(const BwdArgs &a, const WinKeyItem &w)
        : h(w.n > 0 ? w.i0 % w.rows.per_head : 0),
          slice(w.bh * (a.H / a.win.Hkv) + (w.n > 0 ? w.i0 / w.rows.per_head : 0)), per_head(w.rows.per_head) {}
    __device__ __forceinline__ void next() {
        if (++h == per_head) {
            h = 0;
            ++slice;
        }
    }
};

// Query slice (batch and query head) of tile i of key slice kv_bh.
__device__ __forceinline__ int win_query_slice(const BwdArgs &a, int kv_bh, const WinRows &rows, int i) {
    return kv_bh * (a.H / a.win.Hkv) + i / rows.per_head;
}

// bit i: query row q0 + i exists and sees key
__device__ __forceinline__ uint32_t seen_by(const BwdArgs &a, int key, int q0) {
    return key < a.win.Nk ? seeing_positions(key, a.win.Nk - a.N + q0, a.win.window, a.win.sinks) & low_bits(a.N - q0) : 0u;
}

// query rows q0 .. q0 + n - 1 all see key
__device__ __forceinline__ bool sees_all(const BwdArgs &a, int key, int q0, int n) {
    const int p0 = a.win.Nk - a.N + q0;
    return key < a.win.Nk && all_seen(p0, p0 + n - 1, key, key, a.win.window, a.win.sinks);
}
#endif

// 5-GEMM comparator backward (bwd_atomic.cu): a.dq is the fp32 accumulator
// (B*H*N*D floats), dq_out the gradient in grad dtype; D = 128 only.
cudaError_t launch_bwd_atomic(const BwdArgs &a, void *dq_out, const CUtensorMap &tq, const CUtensorMap &tk,
                              const CUtensorMap &tv, const CUtensorMap &tdo, cudaStream_t s);

// Decode (few query rows against a long key range), split over the keys.
constexpr int kNumSms = 152;  // GB300; used only when the device's own SM count cannot be read

struct DecodeArgs {
    const void *q, *k, *v;  // q [B, H, n_q, D]; k, v [B, H, N, D]; bf16
    void *o;                // [B, H, n_q, D] bf16
    float *lse;             // [B, H, n_q]
    float *workspace;       // O, m, l partials of every key chunk (decode_workspace_bytes)
    int B, H, n_q, N, D;
    int splits, chunk;      // key chunks per (batch, head), keys per chunk
    float scale_log2;
    int causal;
};

int decode_max_rows(int D);
// The key-chunk split (and so the workspace size) depends on the device's SM count.
void decode_split(int B, int H, int n_q, int N, int D, int num_sms, int *splits, int *chunk);
size_t decode_workspace_bytes(int B, int H, int n_q, int N, int D, int num_sms);
cudaError_t launch_decode(const DecodeArgs &a, cudaStream_t s);

// Fixed scratch of fa_decode_noalloc (static device storage in decode.cu).
constexpr size_t kDecodeScratchBytes = size_t(16) << 20;
// Device address of the current device's scratch; the first call on a device
// looks it up (cudaGetSymbolAddress), later calls return the cached address.
cudaError_t decode_static_scratch(float **ptr);

// Tensor maps for one [B*H, N, D] bf16 tensor, box = {64, rows, 1}, 128-byte swizzle.
struct TmaPair {
    CUtensorMap map;
};

cudaError_t launch_fwd_f32(const FwdArgs &a, cudaStream_t s);
// `to`: O's tensor map (bf16, 64-column boxes of 128 rows, 128-byte swizzle), for the kernels whose
// epilogue stores O by TMA
cudaError_t launch_fwd_bf16(const FwdArgs &a, const CUtensorMap &tq, const CUtensorMap &tk,
                            const CUtensorMap &tv, const CUtensorMap &to, cudaStream_t s);
cudaError_t launch_fwd_bf16_pair(const FwdArgs &a, const CUtensorMap &tq, const CUtensorMap &tk,
                                 const CUtensorMap &tv, const CUtensorMap &to, cudaStream_t s);
// fwd_bf16_duo.cu: D = 64, the two-tile persistent forward with one issuer warp and one P buffer per tile
cudaError_t launch_fwd_bf16_duo(const FwdArgs &a, const CUtensorMap &tq, const CUtensorMap &tk,
                                const CUtensorMap &tv, cudaStream_t s);
// The dQ kernels also take O's tensor map (128-row boxes; its tile is staged for D_i = rowsum(dO * O))
// and dQ's (grad dtype, 128-byte boxes of 128 rows, 128-byte swizzle: the TMA stores of the epilogue).
cudaError_t launch_bwd_dq(const BwdArgs &a, const CUtensorMap &tq, const CUtensorMap &tk,
                          const CUtensorMap &tv, const CUtensorMap &tdo, const CUtensorMap &to,
                          const CUtensorMap &tdq, cudaStream_t s,
                          bool win = false, bool behind = false);
// bwd_dq_k128.cu: the dQ kernel for D = 64 with 128-row K / V tiles (TMA boxes of 128 rows)
cudaError_t launch_bwd_dq_k128(const BwdArgs &a, const CUtensorMap &tq, const CUtensorMap &tk,
                               const CUtensorMap &tv, const CUtensorMap &tdo, const CUtensorMap &to,
                               const CUtensorMap &tdq, cudaStream_t s);
// The dK/dV kernels also take dK's and dV's tensor maps (grad dtype, 128-byte boxes of 128 rows, 128-byte
// swizzle: the TMA stores of the epilogue).
// bwd_dkdv_q128.cu: the dK/dV kernel for D = 64 with 128-row Q / dO tiles (TMA boxes of 128 rows)
cudaError_t launch_bwd_dkdv_q128(const BwdArgs &a, const CUtensorMap &tq, const CUtensorMap &tk,
                                 const CUtensorMap &tv, const CUtensorMap &tdo, const CUtensorMap &tdk,
                                 const CUtensorMap &tdv, cudaStream_t s);
cudaError_t launch_bwd_dkdv(const BwdArgs &a, const CUtensorMap &tq, const CUtensorMap &tk,
                            const CUtensorMap &tv, const CUtensorMap &tdo, const CUtensorMap &tdk,
                            const CUtensorMap &tdv, cudaStream_t s,
                          const CUtensorMap *parts = nullptr);
// Windowed dQ.  D_i of the rows at the first kExactDelta positions comes from win_delta.cu, launched before it (behind:
// the dQ kernel is that one's programmatic dependent).
cudaError_t launch_win_delta(const BwdArgs &a, cudaStream_t s);
cudaError_t launch_win_dq(const BwdArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                          const CUtensorMap &tdo, const CUtensorMap &to, const CUtensorMap &tdq, int num_sms,
                          bool behind, cudaStream_t s);
cudaError_t launch_win_dq_k128(const BwdArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                          const CUtensorMap &tdo, const CUtensorMap &to, const CUtensorMap &tdq, int num_sms,
                          bool behind, cudaStream_t s);
// Windowed dK/dV.  behind: launched as the programmatic dependent of the dQ kernel before it on the stream (D <= 128);
// parts[0], parts[1] are the tensor maps of the sink tiles' fp32 partials of dK and dV
// ([part][128][D], 32-column boxes); launch_sink_sum adds them.
cudaError_t launch_win_dkdv(const BwdArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                            const CUtensorMap &tdo, const CUtensorMap &tdk, const CUtensorMap &tdv,
                            const CUtensorMap *parts, int num_sms, bool behind, cudaStream_t s);
cudaError_t launch_sink_sum(const BwdArgs &a, const float *part_dk, const float *part_dv, cudaStream_t s);
// The chunks of the rows behind few sinks, launched behind the dK/dV kernel (win_sinks.cu).
cudaError_t launch_win_sinks(const BwdArgs &a, const CUtensorMap &tq, const CUtensorMap &tdo, float *part_dk, float *part_dv,
                             cudaStream_t s);
cudaError_t launch_selftest_timeout(int *status, int limit_us, cudaStream_t s);

// Head dimension a bf16 kernel is built for: the smallest of 64, 128, 192, 256 that holds D.  Any
// D that is a multiple of 8 (so a row is a whole number of 16-byte units) runs on that kernel: the
// TMA loads a 64-column panel that reaches past D with zeros, which add nothing to a score or an
// output column, and the kernels store only the D real columns (row stride D).
inline int kernel_head_dim(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : D <= 192 ? 192 : 256; }

// K/V ring depth of the forward kernel of width D (a template argument of its launch).
constexpr int fwd_nslot(int D) {
    return D == 64 ? kFwdSpecs[0].nslot : D == 128 ? kFwdSpecs[1].nslot : D == 192 ? kFwdSpecs[2].nslot
                                                                                     : kFwdSpecs[3].nslot;
}

inline int fwd_block_n(int D) {
    for (const auto &sp : kFwdSpecs)
        if (sp.D == D) return sp.BN;
    return 0;
}

}  // namespace fa
