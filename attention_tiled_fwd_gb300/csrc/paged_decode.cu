// paged_decode.cu -- attention of a few new rows per sequence against its pages.
//
// Row r of a key head's R = (Hq / Hkv) n_q sits at position len - n_q + r % n_q and sees key j iff j <= p and
// (j < sinks or j > p - window).  One warp a row: a lane holds D / 32 channels, the scores are added over the warp, and the
// softmax runs online in base 2.
#include "fa_internal.h"
#include "paged.cuh"
#include "sm100_ptx.cuh"
#include <cuda_fp16.h>

namespace fa {
namespace {

template <int D, bool FOUR>
__device__ __forceinline__ float cached(const PagedDecodeArgs &a, const uint8_t *pages, bool value, int page, int h, int j, int c) {
    if (page < 0) return 0.f;
    if constexpr (!FOUR) {
        return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(pages + a.pool.at(page, h, j, 2 * D))[c]);
    } else {
        using U = Unit4<D>;
        const uint8_t *unit = pages + a.pool.at(page, h, j & ~15, 9 * D / 16);
        const int u = j & 15, g = c / 32;
        const int word = value ? U::word(u >> 3, g, 4 * (c % 32 / 4) + (u & 7) / 2) : U::word(u >> 3, g, 4 * (u & 7) + c % 32 / 8);
        const int nibble = value ? 4 * (u & 1) + c % 4 : c % 8;
        const int code = reinterpret_cast<const uint32_t *>(unit)[word] >> (4 * nibble) & 15;
        const int scale = value ? U::v_scale(u, g) : U::k_scale(u, g);
        return (code - 8) * __half2float(reinterpret_cast<const __half *>(unit + U::kCodes)[scale]);
    }
}

template <int D, bool FOUR>
__global__ void __launch_bounds__(32) paged_decode_kernel(PagedDecodeArgs a) {
    constexpr int kOwn = D / 32;
    const int r = blockIdx.x, h = blockIdx.y, b = blockIdx.z, lane = threadIdx.x;
    const int len = a.lens ? max(0, min(a.pool.capacity(), a.lens[b])) : a.pool.capacity();
    const int pos = len - a.n_q + r % a.n_q;
    const size_t row = ((size_t)b * a.pool.Hkv + h) * a.R + r;
    float q[kOwn], o[kOwn], m = -INFINITY, l = 0.f;
    for (int i = 0; i < kOwn; ++i) {  // scaled at once: the product of a huge q with a key may not fit, where the score does
        q[i] = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.q)[row * D + lane + 32 * i]) * a.scale_log2;
        o[i] = 0.f;
    }
    for (int j = 0; j <= pos; ++j) {
        if (j >= a.sinks && j <= pos - a.window) {
            j = pos - a.window;
            continue;
        }
        const int page = a.pool.page_of(b, j);
        if (page < 0 && lane == 0) record_failure(a.status, kErrPage, 0);
        float s = 0.f;
        for (int i = 0; i < kOwn; ++i) s = fmaf(q[i], cached<D, FOUR>(a, a.pool.k, false, page, h, j, lane + 32 * i), s);
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        const float mn = fmaxf(m, s), f = m == mn ? 1.f : ex2_approx(m - mn), p = ex2_approx(s - mn);
        l = fmaf(l, f, p);
        m = mn;
        for (int i = 0; i < kOwn; ++i) o[i] = fmaf(o[i], f, p * cached<D, FOUR>(a, a.pool.v, true, page, h, j, lane + 32 * i));
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    for (int i = 0; i < kOwn; ++i) static_cast<__nv_bfloat16 *>(a.o)[row * D + lane + 32 * i] = __float2bfloat16_rn(o[i] * inv);
    if (lane == 0) a.lse[row] = (m + __log2f(l)) * 0.69314718055994531f;
}

template <int D>
cudaError_t launch(const PagedDecodeArgs &a, bool four, cudaStream_t s) {
    const dim3 grid(a.R, a.pool.Hkv, a.B);
    if (four)
        paged_decode_kernel<D, true><<<grid, 32, 0, s>>>(a);
    else
        paged_decode_kernel<D, false><<<grid, 32, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_decode(const PagedDecodeArgs &a, bool four, cudaStream_t s) {
    switch (a.D) {
        case 64: return launch<64>(a, four, s);
        case 128: return launch<128>(a, four, s);
        case 256: return launch<256>(a, four, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace fa
