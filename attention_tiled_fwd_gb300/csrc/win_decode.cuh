// win_decode.cuh -- launch interface of the grouped-head decode kernels (win_decode.cu).
#pragma once
#include "win.cuh"

namespace fa {

struct WinDecodeArgs {
    const void *q;     // [B, Hkv, R, D] bf16, R = (Hq / Hkv) n_q: the caller's [B, Hq, n_q, D]
    const int *lens;   // [B] keys each sequence holds (clamped to [0, N]); null: N
    void *o;           // [B, Hkv, R, D] bf16
    float *lse;        // [B, Hkv, R]
    int B, Hkv, R, n_q, N, D;
    int window, sinks;
    float scale_log2;
    int *status;
    int splits;        // CTAs a sequence's tiles are dealt to
    float *part_o;     // partials [row][splits][D]
    float2 *part_ml;   // [row][splits]
    // cluster: the splits of a row tile are a cluster (2 to 8 CTAs), which joins their partials through distributed
    // shared memory and writes o and lse; nothing else is launched
    int cluster;
    // join (splits = 1): instead of a partial, each CTA joins its rows with the prefix's partials (none: parts.o null) and
    // writes o and lse
    int join;
    PrefixParts parts;
    int behind;  // launched as the programmatic dependent of the launch that writes the prefix's partials
};

// CTAs per (sequence, key head, row tile) for caches that need up to `tiles` tiles.
int win_decode_splits(int B, int Hkv, int R, int tiles, int D, int num_sms);
int win_decode_tile_keys();
// The same where the splits of a row tile form a cluster, or 0 where more of them than it holds are worth a second launch.
int win_decode_cluster(int splits, int tiles);
// SMs that all CTAs of such a launch take at once.
int win_decode_sms(int B, int Hkv, int R, int splits, int D);
cudaError_t launch_win_decode(const WinDecodeArgs &a, const CUtensorMap &tk, const CUtensorMap &tv, cudaStream_t s);
// O and LSE of every row from its a.splits partials and the prefix's (parts.o null: none); a dependent launch.
cudaError_t launch_win_join(const WinDecodeArgs &a, const PrefixParts &parts, cudaStream_t s);

}  // namespace fa
