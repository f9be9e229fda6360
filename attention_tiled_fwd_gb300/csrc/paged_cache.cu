// paged_cache.cu -- rows into a paged cache (rotated by their positions, bf16 or 4 bits), and out of it again.
//
// Rotation: channels (a, b) of a pair turn by the angle of the row's position, a cos - b sin and b cos + a sin, and are
// rounded to bf16 once: sums of two products whose fp32 result lies so near to the border of two bf16 values that its error
// matters (one in some thousands) are computed again with the products' and the sum's rounding errors.  So the rows do not
// depend on the order of the operations, and 4-bit codes, which would turn a last bit into a step, are those of the
// definition.
// 4 bits: scale = fp16(max |y| / 7) of 32 channels of the bf16 row y, code = 8 + y fp32(1 / scale), rounded to even (one
// FMA onto 1.5 2^23, so the product is not rounded first) and clamped to 1 .. 15.  Groups with an infinity or a NaN get a
// NaN scale; a scale past fp16's largest stays there.
//
// What bounds them.  Rows of bf16 into pages: HBM, less the start and the end of one launch: 4 x 4096 rows of 16/4 heads of 128
// 36 us, 5.8 TB/s; 8 x 2048 rows of 32/8 heads 67 us, 6.1 TB/s; without a rotation 6.4 TB/s.  4-bit rows, 71 % of a copy's rate: waits for
// loads (a warp's one task is a chain of length, rows and cosines, and page, with 43 % of the warps that an SM can have), on top of the
// instructions of rounding and packing (issue slots 72 %): the 4 x 4096 rows 38 us, 4.8 TB/s.  One token: a launch and three reads that wait on one
// another (length, page, row), 3.4 us for 64 sequences.  Gather: HBM: 4 sequences of 20000 to 32768 keys of 8 heads in 4 bits
// 85 us, 6.5 TB/s.
// Not kept (append of 2 x 2000 rows of 32/8 heads in 4 bits and a gather of 2 x 9000 to 16384 take 45.4 us): a lane with both halves
// of the pairs (nothing exchanged, fp32 pairs; 46.8 us); 4-bit rows of several heads in turn (45.9 us with two, 47.9 with four);
// 40 warps an SM with 48 registers (45.9 us, and 40 us for the 4 x 4096 rows of bf16).
#include "fa_internal.h"
#include "paged.cuh"
#include "sm100_ptx.cuh"
#include <algorithm>
#include <cuda_fp16.h>

namespace fa {
namespace {

constexpr int kThreads = 128;  // (append of 4 x 4096 rows, of 2 x 2000 in 4 bits with its gather: 37.0, 45.4 us; with 256 38.0, 46.7)
constexpr int kHeadsPerLane = 4;  // rows of one token that a lane turns with the same cosines

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ uint32_t word_of(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// a c + b s rounded to fp32 so that rounding that to bf16 is rounding the exact sum: TwoSum of the products with their
// errors (Knuth; Dekker), and a sum that lies halfway between two bf16 values is moved one step to its side.
__device__ __forceinline__ float turn_exact(float a, float c, float b, float s) {
    const float p = __fmul_rn(a, c), pe = __fmaf_rn(a, c, -p);
    const float w = __fmul_rn(b, s), we = __fmaf_rn(b, s, -w);
    const float h = __fadd_rn(p, w), bb = __fsub_rn(h, p);
    const float he = __fadd_rn(__fsub_rn(p, __fsub_rn(h, bb)), __fsub_rn(w, bb));
    const float t = __fadd_rn(he, __fadd_rn(pe, we));
    const float y = __fadd_rn(h, t), rest = __fsub_rn(t, __fsub_rn(y, h));
    const uint32_t bits = __float_as_uint(y);
    if (!(fabsf(y) < INFINITY)) return __fmaf_rn(a, c, w);
    if ((bits & 0xffffu) == 0x8000u && rest != 0.f) return __uint_as_float(bits + ((rest > 0.f) == (y > 0.f) ? 1 : -1));
    return y;
}

constexpr float kSlack = 0x1.00001p-24f;

// Two channels of a chunk that has one of those: the sums that do not round alike are computed again.
__device__ __noinline__ uint32_t turn_pair(uint32_t xa, uint32_t xb, float c0, float c1, float s0, float s1) {
    const float w0 = bf_lo(xb) * s0, w1 = bf_hi(xb) * s1, v0 = fmaf(bf_lo(xa), c0, w0), v1 = fmaf(bf_hi(xa), c1, w1);
    const float e0 = fabsf(v0) + fabsf(w0), e1 = fabsf(v1) + fabsf(w1);
    const uint32_t y = pack_bf16x2(__fmaf_ru(e0, kSlack, v0), __fmaf_ru(e1, kSlack, v1));
    if (y == pack_bf16x2(__fmaf_rd(e0, -kSlack, v0), __fmaf_rd(e1, -kSlack, v1))) return y;
    return pack_bf16x2(turn_exact(bf_lo(xa), c0, bf_lo(xb), s0), turn_exact(bf_hi(xa), c1, bf_hi(xb), s1));
}

// The rotation of a lane's 8 channels: its own times cos plus their partners' times (signed) sin.
template <bool INTERLEAVED>
struct Turn {
    float c[8], s[8];
    bool on;
    int partner;  // lane offset of the partners' chunk, 0: neighbours within the chunk

    // chunk `cl` of a row at position p
    __device__ __forceinline__ void load(const AppendArgs &a, int p, int cl) {
        on = 8 * cl < a.rot;
        partner = 0;
        if (!on) return;
        const int half = a.rot / 2;
        const float *cs = a.cos + (size_t)p * half, *sn = a.sin + (size_t)p * half;
        if constexpr (INTERLEAVED) {
            const float4 x = *reinterpret_cast<const float4 *>(cs + 4 * cl), y = *reinterpret_cast<const float4 *>(sn + 4 * cl);
            c[0] = c[1] = x.x, c[2] = c[3] = x.y, c[4] = c[5] = x.z, c[6] = c[7] = x.w;
            s[0] = -y.x, s[1] = y.x, s[2] = -y.y, s[3] = y.y, s[4] = -y.z, s[5] = y.z, s[6] = -y.w, s[7] = y.w;
            return;
        }
        const bool low = 8 * cl < half;
        const int at = low ? 8 * cl : 8 * cl - half;
        partner = low ? half / 8 : -(half / 8);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 x = *reinterpret_cast<const float4 *>(cs + at + 4 * i), y = *reinterpret_cast<const float4 *>(sn + at + 4 * i);
            c[4 * i] = x.x, c[4 * i + 1] = x.y, c[4 * i + 2] = x.z, c[4 * i + 3] = x.w;
            s[4 * i] = low ? -y.x : y.x, s[4 * i + 1] = low ? -y.y : y.y, s[4 * i + 2] = low ? -y.z : y.z, s[4 * i + 3] = low ? -y.w : y.w;
        }
    }

    // All lanes of the warp take part.
    __device__ __forceinline__ uint4 apply(const uint4 &x, int lane) const {
        uint4 o;
        const int from = lane + partner;
        if constexpr (INTERLEAVED) {
            o = make_uint4(x.x >> 16 | x.x << 16, x.y >> 16 | x.y << 16, x.z >> 16 | x.z << 16, x.w >> 16 | x.w << 16);
        } else {
            o.x = __shfl_sync(0xffffffffu, x.x, from);
            o.y = __shfl_sync(0xffffffffu, x.y, from);
            o.z = __shfl_sync(0xffffffffu, x.z, from);
            o.w = __shfl_sync(0xffffffffu, x.w, from);
        }
        if (!on) return x;
        uint32_t y[4], near = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t xa = word_of(x, i), xb = word_of(o, i);
            const float w0 = bf_lo(xb) * s[2 * i], w1 = bf_hi(xb) * s[2 * i + 1];
            const float v0 = fmaf(bf_lo(xa), c[2 * i], w0), v1 = fmaf(bf_hi(xa), c[2 * i + 1], w1);
            // v is off by half a step of itself and of w at most, 2^-24 (|v| + |w|): does all of that round alike?
            const float e0 = fabsf(v0) + fabsf(w0), e1 = fabsf(v1) + fabsf(w1);
            y[i] = pack_bf16x2(__fmaf_ru(e0, kSlack, v0), __fmaf_ru(e1, kSlack, v1));
            near |= y[i] ^ pack_bf16x2(__fmaf_rd(e0, -kSlack, v0), __fmaf_rd(e1, -kSlack, v1));
        }
        // (zeros end up here, as 0 and -0; rows of padding need no more)
        if (near && ((x.x | x.y | x.z | x.w | o.x | o.y | o.z | o.w) & 0x7fff7fffu)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = turn_pair(word_of(x, i), word_of(o, i), c[2 * i], c[2 * i + 1], s[2 * i], s[2 * i + 1]);
        }
        return make_uint4(y[0], y[1], y[2], y[3]);
    }
};

// The new rows of sequence b: positions [first, len).  A row past the capacity has no page, and no cosines either.
struct NewRows {
    int first, len, start;  // start: the position of row 0 (may be below 0)
    __device__ __forceinline__ NewRows(const AppendArgs &a, int b) {
        len = max(0, min(a.lens[b], a.pool.capacity() + a.n));  // (past that no row has a page: sums stay within 32 bits)
        const int n = a.counts ? max(0, min(a.n, a.counts[b])) : a.n;
        start = len - a.n;
        first = max(0, len - n);
    }
};

// Rows of one token: lane `cl` of a row's D / 8 holds 8 channels, of kHeadsPerLane heads in turn, a block of heads.  `part`: `per`
// blocks of q, then (bf16 pages) a block of k and v.
template <int D, bool FOUR, bool INTERLEAVED>
__device__ __forceinline__ void token_rows(const AppendArgs &a, int b, int i, int part, int per) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kBlock = kRows * kHeadsPerLane;
    const int lane = threadIdx.x & 31, cl = lane % kLanes, sub = lane / kLanes;
    const int q_parts = (a.Hq + per * kBlock - 1) / (per * kBlock);
    const bool is_q = FOUR || part < q_parts;
    const int heads = is_q ? a.Hq : a.pool.Hkv;
    int h = (is_q ? part * per : part - q_parts) * kBlock + sub;  // this lane's first head of a block
    auto fetch = [&](uint4(&x)[kHeadsPerLane], const void *t, const long long *st) {
        const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(t) + b * st[0] + h * st[1] + i * st[2] + 8 * cl;
        const long long step = kRows * st[1];
#pragma unroll
        for (int u = 0; u < kHeadsPerLane; ++u, src += step) {
            x[u] = make_uint4(0, 0, 0, 0);
            if (h + u * kRows < heads) x[u] = __ldg(reinterpret_cast<const uint4 *>(src));
        }
    };
    uint4 x[kHeadsPerLane];  // (rows that are not new too: the loads need not wait for the lengths)
    fetch(x, is_q ? a.q : a.k, is_q ? a.sq : a.sk);
    const NewRows rows(a, b);
    const int p = rows.start + i;
    const bool there = p >= rows.first && p < a.pool.capacity();
    Turn<INTERLEAVED> turn;
    turn.on = false, turn.partner = 0;
    if (there && a.rot > 0) turn.load(a, p, cl);
    if (is_q) {
        uint4 *to = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.q_out) + (((size_t)b * a.Hq + h) * a.n + i) * D) + cl;
        const size_t step = (size_t)kRows * a.n * (D / 8);
        for (int block = 0;;) {
#pragma unroll
            for (int u = 0; u < kHeadsPerLane; ++u, to += step) {
                if (h - sub + u * kRows >= heads) return;
                const uint4 y = !there ? make_uint4(0, 0, 0, 0) : a.rot > 0 ? turn.apply(x[u], lane) : x[u];
                if (h + u * kRows < heads) *to = y;
            }
            if (++block == per) return;
            h += kBlock;
            fetch(x, a.q, a.sq);
        }
    } else if constexpr (!FOUR) {
        if (p < rows.first) return;
        const int page = there ? a.pool.page_of(b, p) : -1;
        if (page < 0) {
            if (lane == 0) record_failure(a.status, kErrPage, 0);
            return;
        }
        uint4 v[kHeadsPerLane];
        fetch(v, a.v, a.sv);
        const size_t at = a.pool.at(page, h, p, 2 * D), step = ((size_t)kRows << a.pool.shift) * (D / 8);
        uint4 *to_k = reinterpret_cast<uint4 *>(a.pool.k + at) + cl, *to_v = reinterpret_cast<uint4 *>(a.pool.v + at) + cl;
#pragma unroll
        for (int u = 0; u < kHeadsPerLane; ++u, to_k += step, to_v += step) {
            if (h - sub + u * kRows >= heads) return;
            const uint4 y = a.rot > 0 ? turn.apply(x[u], lane) : x[u];
            if (h + u * kRows < heads) *to_k = y, *to_v = v[u];
        }
    }
}

__device__ __forceinline__ uint32_t max_u2(uint32_t a, uint32_t b) {  // of pairs of 16-bit integers
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// 8 channels of a row in 4 bits: its 8 codes, the lowest channel in the lowest bits, and the scale of the 32 channels that
// its four lanes share.
__device__ __forceinline__ uint32_t quantise(const uint4 &y, __half *scale) {
    constexpr uint32_t kAbs = 0x7fff7fffu, kMagic = 0x4B400000u;  // 1.5 2^23
    uint32_t most = max_u2(max_u2(y.x & kAbs, y.y & kAbs), max_u2(y.z & kAbs, y.w & kAbs));  // magnitudes order as integers, NaN above all
    most = max_u2(most, __shfl_xor_sync(0xffffffffu, most, 1));
    most = max_u2(most, __shfl_xor_sync(0xffffffffu, most, 2));
    most = max(most << 16, most & 0xffff0000u);
    // a seventh, its error taken off: exact where it is a number of fp32, so ties of fp16 are ties
    const float m = __uint_as_float(most), near = m * (1.f / 7.f), seventh = fmaf(fmaf(-7.f, near, m), 1.f / 7.f, near);
    const __half s = most < 0x7f800000u ? __float2half_rn(fminf(seventh, 65504.f)) : __ushort_as_half(0x7fff);
    const float f = __half2float(s), inverse = f > 0.f ? __frcp_rn(f) : 0.f;  // (NaN: codes do not matter)
    *scale = s;
    float v[8];
    const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f2_unpack(f2_fma(f2_pack(bf_lo(w[i]), bf_hi(w[i])), f2_pack(inverse, inverse), f2_pack(12582920.f, 12582920.f)), v[2 * i], v[2 * i + 1]);
    // a normal scale is at most 2^-11 too small, so 8 + step is in 1 .. 15
    if ((uint32_t)__half_as_ushort(s) - 0x0400u >= 0x7bffu - 0x0400u) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fminf(fmaxf(v[i], 12582913.f), 12582927.f);
    }
    uint32_t codes = 0, magic = 0;
#pragma unroll
    for (int i = 7; i >= 0; --i) {
        codes = codes * 16 + __float_as_uint(v[i]);
        magic = magic * 16 + kMagic;
    }
    return codes - magic;
}

// 4-bit rows of a head's keys or values: a lane holds 8 channels of an even position and of the odd one behind it, so a warp
// the 64 / (D / 8) positions of a block of them (never of two units).
template <int D, bool INTERLEAVED>
__device__ __forceinline__ void unit_rows(const AppendArgs &a, int b, int block, int part) {
    using U = Unit4<D>;
    constexpr int kLanes = D / 8, kBlock = 64 / kLanes;
    const int lane = threadIdx.x & 31, cl = lane % kLanes, sub = lane / kLanes;
    const bool key = part < a.pool.Hkv;
    const int h = key ? part : part - a.pool.Hkv;
    const NewRows rows(a, b);
    const int p0 = (rows.first / kBlock + block) * kBlock + 2 * sub;  // this lane's even position
    if (p0 - 2 * sub >= rows.len || rows.first >= rows.len) return;
    const long long *st = key ? a.sk : a.sv;
    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(key ? a.k : a.v) + b * st[0] + h * st[1] + (p0 - rows.start) * st[2] + 8 * cl;
    uint4 x[2];
    bool there[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        there[e] = p0 + e >= rows.first && p0 + e < rows.len;
        x[e] = there[e] ? __ldg(reinterpret_cast<const uint4 *>(src + e * st[2])) : make_uint4(0, 0, 0, 0);
    }
    const int page = p0 < a.pool.capacity() ? a.pool.page_of(b, p0) : -1;
    if (page < 0) {
        if (lane == 0) record_failure(a.status, kErrPage, 0);
        return;
    }
    uint32_t codes[2];
    __half scale[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        if (key && a.rot > 0) {
            Turn<INTERLEAVED> turn;
            turn.on = false, turn.partner = 0;
            if (there[e]) turn.load(a, p0 + e, cl);
            x[e] = turn.apply(x[e], lane);
        }
        codes[e] = quantise(x[e], &scale[e]);
    }
    const int u = p0 & (kUnit - 1), g = cl / 4, t = cl % 4;
    uint8_t *to = (key ? a.pool.k : a.pool.v) + a.pool.at(page, h, p0 - u, 9 * D / 16);
    __half *scales = reinterpret_cast<__half *>(to + U::kCodes);
    if (key) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (!there[e]) continue;
            reinterpret_cast<uint32_t *>(to)[U::word(u >> 3, g, 4 * ((u + e) & 7) + t)] = codes[e];
            if (t == 0) scales[U::k_scale(u + e, g)] = scale[e];
        }
        return;
    }
    // channels 8 t .. of the group: lanes' fourths 2 t and 2 t + 1
    uint32_t *w0 = reinterpret_cast<uint32_t *>(to) + U::word(u >> 3, g, 8 * t + (u & 7) / 2);
    uint32_t *w1 = reinterpret_cast<uint32_t *>(to) + U::word(u >> 3, g, 8 * t + 4 + (u & 7) / 2);
    if (there[0] && there[1]) {
        *w0 = __byte_perm(codes[0], codes[1], 0x5410);
        *w1 = __byte_perm(codes[0], codes[1], 0x7632);
    } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (!there[e]) continue;
            reinterpret_cast<uint16_t *>(w0)[e] = (uint16_t)codes[e];
            reinterpret_cast<uint16_t *>(w1)[e] = (uint16_t)(codes[e] >> 16);
        }
    }
    if (t == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (there[e]) scales[U::v_scale(u + e, g)] = scale[e];
    }
}

// blockIdx.y: the sequence.  Along x the rows of tokens, then the 4-bit rows, a warp each.
template <int D, bool FOUR, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 8)
    paged_append_kernel(AppendArgs a, FastDiv parts, FastDiv unit_parts, int row_tasks, int unit_tasks, int per) {
    const int task = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), b = blockIdx.y;
    if (task < row_tasks) {
        const int i = parts.div(task);
        token_rows<D, FOUR, INTERLEAVED>(a, b, i, task - i * parts.d, per);
    } else if constexpr (FOUR) {
        const int unit = task - row_tasks;
        if (unit >= unit_tasks) return;
        const int block = unit_parts.div(unit);
        unit_rows<D, INTERLEAVED>(a, b, block, unit - block * unit_parts.d);
    }
}

template <int D, bool FOUR, bool INTERLEAVED>
cudaError_t launch_append(const AppendArgs &a, cudaStream_t s) {
    constexpr int kBlock = 32 / (D / 8) * kHeadsPerLane, kWarps = kThreads / 32, kPositions = 64 / (D / 8);
    const int Hkv = a.pool.Hkv, q_blocks = (a.Hq + kBlock - 1) / kBlock;
    // A warp takes up to four blocks of q where that leaves 32 warps an SM twice over: what it does once (lengths, angles, addresses)
    // is as much as two blocks' rotation (4 x 4096 rows of 16/4 heads, before other steps: 41 us with one block, 38 with two).
    const long long warps = (long long)a.B * a.n * q_blocks;
    const int per = (int)std::max(1ll, std::min<long long>(std::min(4, q_blocks), warps / (64 * kNumSms)));
    const int parts = (q_blocks + per - 1) / per + (FOUR ? 0 : (Hkv + kBlock - 1) / kBlock);
    const int blocks = a.n == 1 ? 1 : (a.n + kPositions - 2) / kPositions + 1;  // of positions that n rows meet at most
    const int row_tasks = a.n * parts, unit_tasks = FOUR ? blocks * 2 * Hkv : 0;
    const dim3 grid((row_tasks + unit_tasks + kWarps - 1) / kWarps, a.B);
    paged_append_kernel<D, FOUR, INTERLEAVED>
        <<<grid, kThreads, 0, s>>>(a, FastDiv(std::max(parts, 1)), FastDiv(2 * Hkv), row_tasks, unit_tasks, per);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_append_d(const AppendArgs &a, bool four, cudaStream_t s) {
    if (a.interleaved) return four ? launch_append<D, true, true>(a, s) : launch_append<D, false, true>(a, s);
    return four ? launch_append<D, true, false>(a, s) : launch_append<D, false, false>(a, s);
}

// One unit of 16 positions of a head's keys or values a warp.
template <int D, bool FOUR>
__global__ void __launch_bounds__(kThreads) paged_gather_kernel(GatherArgs a, int units, long long tasks) {
    const int lane = threadIdx.x & 31;
    const long long task = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (task >= tasks) return;
    const int Hkv = a.pool.Hkv;
    const unsigned bh = (unsigned)(task / units);  // (up to 2^32)
    const int p0 = (int)(task % units) * kUnit, which = bh % 2, h = bh / 2 % Hkv, b = bh / 2 / Hkv;
    const int len = min(a.lens ? max(0, min(a.pool.capacity(), a.lens[b])) : a.pool.capacity(), a.rows);
    if (p0 >= len) return;
    const int n = min(kUnit, len - p0);
    const int page = a.pool.page_of(b, p0);
    if (page < 0 && lane == 0) record_failure(a.status, kErrPage, 0);
    const uint8_t *pages = which ? a.pool.v : a.pool.k;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(which ? a.v : a.k) + (((size_t)b * Hkv + h) * a.rows + p0) * D;
    if constexpr (!FOUR) {
        constexpr int kChunks = D / 8;
        const uint4 *src = reinterpret_cast<const uint4 *>(pages + a.pool.at(max(page, 0), h, p0, 2 * D));
        uint4 x[kUnit * kChunks / 32];
#pragma unroll
        for (int i = 0; i < kUnit * kChunks / 32; ++i) {
            const int c = i * 32 + lane;
            x[i] = page >= 0 && c < n * kChunks ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kUnit * kChunks / 32; ++i) {
            const int c = i * 32 + lane;
            if (c < n * kChunks) reinterpret_cast<uint4 *>(out)[c] = x[i];
        }
    } else {
        using U = Unit4<D>;
        const uint8_t *unit = pages + a.pool.at(max(page, 0), h, p0, 9 * D / 16);
        const __half *scales = reinterpret_cast<const __half *>(unit + U::kCodes);
        auto value = [](uint32_t w, int i, float s) { return ((int)(w >> (4 * i) & 15) - 8) * s; };
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int g = 0; g < U::kGroups; ++g) {
                const uint32_t w = page >= 0 ? __ldg(reinterpret_cast<const uint32_t *>(unit) + U::word(half, g, lane)) : 0x88888888u;
                if (which == 0) {
                    const int u = 8 * half + lane / 4;
                    if (u >= n) continue;
                    const float s = page >= 0 ? __half2float(scales[U::k_scale(u, g)]) : 0.f;
                    reinterpret_cast<uint4 *>(out + u * D + 32 * g)[lane % 4] =
                        make_uint4(pack_bf16x2(value(w, 0, s), value(w, 1, s)), pack_bf16x2(value(w, 2, s), value(w, 3, s)),
                                   pack_bf16x2(value(w, 4, s), value(w, 5, s)), pack_bf16x2(value(w, 6, s), value(w, 7, s)));
                } else {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int u = 8 * half + 2 * (lane % 4) + e;
                        if (u >= n) continue;
                        const float s = page >= 0 ? __half2float(scales[U::v_scale(u, g)]) : 0.f;
                        reinterpret_cast<uint2 *>(out + u * D + 32 * g)[lane / 4] =
                            make_uint2(pack_bf16x2(value(w, 4 * e, s), value(w, 4 * e + 1, s)),
                                       pack_bf16x2(value(w, 4 * e + 2, s), value(w, 4 * e + 3, s)));
                    }
                }
            }
        }
    }
}

template <int D, bool FOUR>
cudaError_t launch_gather(const GatherArgs &a, cudaStream_t s) {
    const int units = (min(a.rows, a.pool.capacity()) + kUnit - 1) / kUnit;
    const long long tasks = (long long)a.B * a.pool.Hkv * 2 * units;
    paged_gather_kernel<D, FOUR><<<(unsigned)((tasks + kThreads / 32 - 1) / (kThreads / 32)), kThreads, 0, s>>>(a, units, tasks);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs &a, bool four, cudaStream_t s) {
    switch (a.D) {
        case 64: return launch_append_d<64>(a, four, s);
        case 128: return launch_append_d<128>(a, four, s);
        case 256: return launch_append_d<256>(a, four, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_paged_gather(const GatherArgs &a, bool four, cudaStream_t s) {
    switch (a.D) {
        case 64: return four ? launch_gather<64, true>(a, s) : launch_gather<64, false>(a, s);
        case 128: return four ? launch_gather<128, true>(a, s) : launch_gather<128, false>(a, s);
        case 256: return four ? launch_gather<256, true>(a, s) : launch_gather<256, false>(a, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace fa
