// fa_api.cu -- the C ABI declared in include/fa.h: argument validation,
// TMA descriptor encoding, and launches on the caller's stream.
//
// Nothing here allocates device memory.  The only device-side state is the
// library's own static storage: the status word below (one int per device),
// which kernels update when a bounded wait runs out, and a ring of work
// counters for the persistent forwards (each zeroed again by the launch that
// used it).
#include "../../include/fa.h"
#include "fa_internal.h"
#include "sm100_ptx.cuh"
#include "win_decode.cuh"

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

namespace fa {

__device__ int g_status_word;

// Work counters (two ints each) of the persistent forwards, handed out in turn, so that launches in
// flight on different streams draw from different counters.
constexpr int kWorkCounters = 1024;
__device__ int g_work_counters[2 * kWorkCounters];

namespace {

constexpr int kMaxDevices = 64;

struct DeviceState {
    bool ready = false;
    int status_code = 0;  // FA_OK or the fa_status of the failed set-up
    int *status_word = nullptr;
    int num_sms = kNumSms;  // the device's SM count (sizes persistent grids)
    long long l2_bytes = 0;  // the device's L2 size (sizes the groups of the causal work order)
    int *work_counters = nullptr;
    std::atomic<unsigned> work_seq{0};
};
DeviceState g_dev[kMaxDevices];
std::mutex g_mu;

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode = nullptr;

// Per-device set-up: architecture check and the status word's device address.
int device_state(int *dev_out, DeviceState **st_out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
    if (dev < 0 || dev >= kMaxDevices) return FA_ERR_DEVICE;
    // Bind the device's primary context to the calling thread: a thread that has made no runtime
    // call yet (a worker thread, autograd's backward thread) has no current context, and the
    // tensor-map encoder is a driver call that needs one.
    if (cudaSetDevice(dev) != cudaSuccess) return FA_ERR_CUDA;
    std::lock_guard<std::mutex> lk(g_mu);
    DeviceState &st = g_dev[dev];
    if (!st.ready) {
        cudaDeviceProp prop;
        if (cudaGetDeviceProperties(&prop, dev) != cudaSuccess) return FA_ERR_CUDA;
        st.num_sms = prop.multiProcessorCount > 0 ? prop.multiProcessorCount : kNumSms;
        st.l2_bytes = prop.l2CacheSize;
        if (!(prop.major == 10 && prop.minor == 3)) {
            st.status_code = FA_ERR_DEVICE;  // kernels are built for sm_103a only
        } else if (cudaGetSymbolAddress(reinterpret_cast<void **>(&st.status_word), g_status_word) != cudaSuccess ||
                   cudaGetSymbolAddress(reinterpret_cast<void **>(&st.work_counters), g_work_counters) !=
                       cudaSuccess) {
            st.status_code = FA_ERR_CUDA;
        } else {
            st.status_code = FA_OK;
        }
        if (!g_encode && st.status_code == FA_OK) {
            cudaDriverEntryPointQueryResult q;
            void *fn = nullptr;
            if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
                    cudaSuccess ||
                q != cudaDriverEntryPointSuccess || !fn)
                st.status_code = FA_ERR_CUDA;
            else
                g_encode = reinterpret_cast<EncodeTiledFn>(fn);
        }
        st.ready = true;
    }
    *dev_out = dev;
    *st_out = &st;
    return st.status_code;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Device-accessible (device or managed memory on the current device).
int check_device_ptr(const void *p) {
    cudaPointerAttributes attr;
    if (cudaPointerGetAttributes(&attr, p) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_DEVICE_PTR;
    }
    if (attr.type != cudaMemoryTypeDevice && attr.type != cudaMemoryTypeManaged) return FA_ERR_DEVICE_PTR;
    return FA_OK;
}

int check_ptrs(std::initializer_list<const void *> ptrs) {
    for (const void *p : ptrs)
        if (!p) return FA_ERR_NULL;
    for (const void *p : ptrs)
        if (!aligned16(p)) return FA_ERR_ALIGN;
    for (const void *p : ptrs) {
        int rc = check_device_ptr(p);
        if (rc != FA_OK) return rc;
    }
    return FA_OK;
}

int check_shape(int B, int H, int N, int D, float scale) {
    if (B < 1 || H < 1 || N < 1 || D < 1) return FA_ERR_SHAPE;
    if (B > 65535 || H > 65535) return FA_ERR_SHAPE;  // grid y / z limits
    if ((long long)B * H * (long long)N > (1ll << 31) - 1) return FA_ERR_SHAPE;
    if (!std::isfinite(scale)) return FA_ERR_SCALE;
    return FA_OK;
}

// [B*H, N, D] bf16 or fp32 tensor, box {128 bytes of a row, rows, 1}, 128-byte swizzle, zero fill out of
// bounds (loads) and clipping (stores).
int encode_3d(CUtensorMap *map, const void *base, int BH, int N, int D, int box_rows, bool f32) {
    const int elt = f32 ? 4 : 2;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)N, (cuuint64_t)BH};
    cuuint64_t strides[2] = {(cuuint64_t)D * elt, (cuuint64_t)N * D * elt};
    cuuint32_t box[3] = {(cuuint32_t)(128 / elt), (cuuint32_t)box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = g_encode(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                          const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

// [slices, rows, D] bf16 tensor whose slices lie slice_rows rows apart, box {64, box_rows, 1}, 128-byte swizzle,
// zero fill out of bounds.
int encode_rows(CUtensorMap *map, const void *base, int slices, int rows, int slice_rows, int D, int box_rows) {
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)rows, (cuuint64_t)slices};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)slice_rows * D * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
                          estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

// [B*H, N, D] bf16 tensor, box {64, rows, 1}, 128-byte swizzle, zero fill out of bounds.
int encode_bf16_3d(CUtensorMap *map, const void *base, int BH, int N, int D, int box_rows) {
    return encode_rows(map, base, BH, N, N, D, box_rows);
}

float log2e() { return 1.4426950408889634f; }

// bf16 head dimensions the tensor-core kernels take: a multiple of 8 (whole 16-byte units per row, as
// the TMA needs for the row stride) up to 256; each runs on the kernel of width kernel_head_dim(D).
bool bf16_head_dim_ok(int D) { return D >= 8 && D <= 256 && D % 8 == 0; }

// SM count of the current device for the host-side size queries, which must also answer without a
// usable device (they make no launch): the GB300 count when it cannot be read.
int current_num_sms() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) !=
                                                  cudaSuccess) {
        cudaGetLastError();
        return kNumSms;
    }
    return sms > 0 ? sms : kNumSms;
}

// Heads per group of the causal work order (tile_order_at).  A launch streams two [N, D] bf16 operands per
// head (K and V, or Q and dO); while those of every head fit in three quarters of L2 the order is the plain
// rank order over all heads, otherwise a group holds as many heads as fit in a quarter of it (at least
// one), so that its operands stay in L2 while the group's CTAs read them.  (Three eighths, a half, five
// eighths and three quarters of L2 measured 0-3 % slower at B=1 H=32 N=32768 D=64 and N=16384 D=128.)
int causal_head_group(const DeviceState &st, int B, int H, int N, int D) {
    const int n_bh = B * H;
    const double per_head = 4.0 * N * D;
    const double l2 = st.l2_bytes > 0 ? (double)st.l2_bytes : 126.0 * (1 << 20);
    if (per_head * n_bh <= 0.75 * l2) return n_bh;
    return std::max(1, std::min(n_bh, (int)(0.25 * l2 / per_head)));
}

// The persistent forwards draw their blocks from a work counter when the causal order runs by groups of
// heads (only drawing in turn balances such a sequence); with one group they use the static deal.
int *forward_work_counter(DeviceState &st, int head_group, int B, int H, int causal) {
    if (!causal || head_group >= B * H) return nullptr;
    return st.work_counters + 2 * (st.work_seq.fetch_add(1, std::memory_order_relaxed) % kWorkCounters);
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" int fa_forward(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H, int N,
                          int D, float scale, int causal, int dtype, void *stream) {
    int rc = check_shape(B, H, N, D, scale);
    if (rc != FA_OK) return rc;
    if (dtype == FA_BF16) {
        if (!bf16_head_dim_ok(D)) return FA_ERR_HEAD_DIM;
    } else if (dtype == FA_F32) {
        if (D % 4 != 0 || D > 256) return FA_ERR_HEAD_DIM;
    } else {
        return FA_ERR_DTYPE;
    }
    rc = check_ptrs({q, k, v, o, lse});
    if (rc != FA_OK) return rc;
    int dev;
    DeviceState *st;
    rc = device_state(&dev, &st);
    if (rc != FA_OK) return rc;

    // The D = 128 kernel deals its blocks statically, and so keeps the plain rank order over all heads: handing
    // its issuer warp drawn blocks measured 10-15 % slower.  The D = 64 kernel draws them (a work counter) when
    // the order runs by groups; the other kernels launch one CTA per tile, which the hardware hands out in turn.
    const int Dk = dtype == FA_BF16 ? kernel_head_dim(D) : 0;
    const int group = Dk == 128 ? B * H : causal_head_group(*st, B, H, N, D);
    FwdArgs a{q, k, v, o, lse, B, H, N, D, scale, scale * log2e(), causal ? 1 : 0, st->status_word, st->num_sms,
              group, nullptr};
    if (Dk == 64) a.work = forward_work_counter(*st, group, B, H, causal);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == FA_F32) {
        e = launch_fwd_f32(a, s);
    } else {
        CUtensorMap tq, tk, tv, to;
        const int bn = fwd_block_n(kernel_head_dim(D));
        if (encode_bf16_3d(&tq, q, B * H, N, D, 128) != FA_OK || encode_bf16_3d(&tk, k, B * H, N, D, bn) != FA_OK ||
            encode_bf16_3d(&tv, v, B * H, N, D, bn) != FA_OK || encode_bf16_3d(&to, o, B * H, N, D, 128) != FA_OK)
            return FA_ERR_CUDA;
        e = launch_fwd_bf16(a, tq, tk, tv, to, s);
    }
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

extern "C" int fa_backward_dq(const void *q, const void *k, const void *v, const void *o, const void *dO,
                              const float *lse, float *delta, void *dq, int B, int H, int N, int D, float scale,
                              int causal, int dtype, int grad_dtype, void *stream) {
    int rc = check_shape(B, H, N, D, scale);
    if (rc != FA_OK) return rc;
    if (dtype != FA_BF16 && dtype != FA_F32) return FA_ERR_DTYPE;
    if (grad_dtype != FA_BF16 && grad_dtype != FA_F32) return FA_ERR_DTYPE;
    if (dtype != FA_BF16) return FA_ERR_DTYPE;  // the split backward runs on bf16 inputs
    if (!bf16_head_dim_ok(D)) return FA_ERR_HEAD_DIM;
    rc = check_ptrs({q, k, v, o, dO, lse, delta, dq});
    if (rc != FA_OK) return rc;
    int dev;
    DeviceState *st;
    rc = device_state(&dev, &st);
    if (rc != FA_OK) return rc;
    BwdArgs a{q, k, v, o, dO, lse, delta, dq, nullptr, nullptr, B, H, N, D, scale, scale * log2e(),
              causal ? 1 : 0, grad_dtype == FA_BF16 ? 1 : 0, st->status_word, causal_head_group(*st, B, H, N, D)};
    CUtensorMap tq, tk, tv, tdo, to, tdq;
    // D <= 64 runs the 128-key-tile kernel (its score products are N = 128 MMAs); wider heads the 64-key one
    const int Dk = kernel_head_dim(D);
    const int kv_rows = Dk == 64 ? 128 : kDqKRows;
    if (encode_bf16_3d(&tq, q, B * H, N, D, 128) != FA_OK ||
        encode_bf16_3d(&tk, k, B * H, N, D, kv_rows) != FA_OK ||
        encode_bf16_3d(&tv, v, B * H, N, D, kv_rows) != FA_OK ||
        encode_bf16_3d(&tdo, dO, B * H, N, D, 128) != FA_OK || encode_bf16_3d(&to, o, B * H, N, D, 128) != FA_OK ||
        encode_3d(&tdq, dq, B * H, N, D, 128, grad_dtype == FA_F32) != FA_OK)
        return FA_ERR_CUDA;
    cudaError_t e = Dk == 64
                        ? launch_bwd_dq_k128(a, tq, tk, tv, tdo, to, tdq, reinterpret_cast<cudaStream_t>(stream))
                        : launch_bwd_dq(a, tq, tk, tv, tdo, to, tdq, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

extern "C" int fa_backward_dkdv(const void *q, const void *k, const void *v, const void *dO, const float *lse,
                                const float *delta, void *dk, void *dv, int B, int H, int N, int D, float scale,
                                int causal, int dtype, int grad_dtype, void *stream) {
    int rc = check_shape(B, H, N, D, scale);
    if (rc != FA_OK) return rc;
    if (dtype != FA_BF16 && dtype != FA_F32) return FA_ERR_DTYPE;
    if (grad_dtype != FA_BF16 && grad_dtype != FA_F32) return FA_ERR_DTYPE;
    if (dtype != FA_BF16) return FA_ERR_DTYPE;
    if (!bf16_head_dim_ok(D)) return FA_ERR_HEAD_DIM;
    rc = check_ptrs({q, k, v, dO, lse, delta, dk, dv});
    if (rc != FA_OK) return rc;
    int dev;
    DeviceState *st;
    rc = device_state(&dev, &st);
    if (rc != FA_OK) return rc;
    BwdArgs a{q, k, v, nullptr, dO, lse, const_cast<float *>(delta), nullptr, dk, dv, B, H, N, D, scale,
              scale * log2e(), causal ? 1 : 0, grad_dtype == FA_BF16 ? 1 : 0, st->status_word,
              causal_head_group(*st, B, H, N, D)};
    CUtensorMap tq, tk, tv, tdo, tdk, tdv;
    // D <= 64 runs the 128-query-tile kernel (its score products are N = 128 MMAs); wider heads the 64-query one
    const int Dk = kernel_head_dim(D);
    const int q_rows = Dk == 64 ? 128 : kDkdvQRows;
    if (encode_bf16_3d(&tq, q, B * H, N, D, q_rows) != FA_OK ||
        encode_bf16_3d(&tk, k, B * H, N, D, 128) != FA_OK || encode_bf16_3d(&tv, v, B * H, N, D, 128) != FA_OK ||
        encode_bf16_3d(&tdo, dO, B * H, N, D, q_rows) != FA_OK ||
        encode_3d(&tdk, dk, B * H, N, D, 128, grad_dtype == FA_F32) != FA_OK ||
        encode_3d(&tdv, dv, B * H, N, D, 128, grad_dtype == FA_F32) != FA_OK)
        return FA_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = Dk == 64 ? launch_bwd_dkdv_q128(a, tq, tk, tv, tdo, tdk, tdv, s)
                             : launch_bwd_dkdv(a, tq, tk, tv, tdo, tdk, tdv, s);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

extern "C" int fa_backward_atomic(const void *q, const void *k, const void *v, const void *o, const void *dO,
                                  const float *lse, float *delta, void *dq, void *dk, void *dv, float *dq_accum,
                                  size_t dq_accum_bytes, int B, int H, int N, int D, float scale, int causal,
                                  int dtype, int grad_dtype, void *stream) {
    int rc = check_shape(B, H, N, D, scale);
    if (rc != FA_OK) return rc;
    if (dtype != FA_BF16 && dtype != FA_F32) return FA_ERR_DTYPE;
    if (grad_dtype != FA_BF16 && grad_dtype != FA_F32) return FA_ERR_DTYPE;
    if (dtype != FA_BF16) return FA_ERR_DTYPE;
    if (D != 128) return FA_ERR_HEAD_DIM;
    rc = check_ptrs({q, k, v, o, dO, lse, delta, dq, dk, dv, dq_accum});
    if (rc != FA_OK) return rc;
    if (dq_accum_bytes < (size_t)B * H * N * D * sizeof(float)) return FA_ERR_WORKSPACE;
    int dev;
    DeviceState *st;
    rc = device_state(&dev, &st);
    if (rc != FA_OK) return rc;
    BwdArgs a{q, k, v, o, dO, lse, delta, dq_accum, dk, dv, B, H, N, D, scale, scale * log2e(),
              causal ? 1 : 0, grad_dtype == FA_BF16 ? 1 : 0, st->status_word, causal_head_group(*st, B, H, N, D)};
    CUtensorMap tq, tk, tv, tdo;
    if (encode_bf16_3d(&tq, q, B * H, N, D, kDkdvQRows) != FA_OK || encode_bf16_3d(&tk, k, B * H, N, D, 128) != FA_OK ||
        encode_bf16_3d(&tv, v, B * H, N, D, 128) != FA_OK || encode_bf16_3d(&tdo, dO, B * H, N, D, kDkdvQRows) != FA_OK)
        return FA_ERR_CUDA;
    cudaError_t e = launch_bwd_atomic(a, dq, tq, tk, tv, tdo, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

namespace {
int check_decode(int B, int H, int n_q, int N, int D, float scale) {
    int rc = check_shape(B, H, N, D, scale);
    if (rc != FA_OK) return rc;
    if (D != 64 && D != 128 && D != 256) return FA_ERR_HEAD_DIM;
    if (n_q < 1 || n_q > decode_max_rows(D) || n_q > N) return FA_ERR_SHAPE;
    if ((long long)B * H * (long long)n_q > (1ll << 31) - 1) return FA_ERR_SHAPE;
    return FA_OK;
}
}  // namespace

extern "C" int fa_decode_workspace_bytes(int B, int H, int n_q, int N, int D, size_t *bytes) {
    if (!bytes) return FA_ERR_NULL;
    int rc = check_decode(B, H, n_q, N, D, 1.f);
    if (rc != FA_OK) return rc;
    *bytes = decode_workspace_bytes(B, H, n_q, N, D, current_num_sms());
    return FA_OK;
}

extern "C" int fa_decode(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H, int n_q,
                         int N, int D, float scale, int causal, void *workspace, size_t workspace_bytes,
                         void *stream) {
    int rc = check_decode(B, H, n_q, N, D, scale);
    if (rc != FA_OK) return rc;
    rc = check_ptrs({q, k, v, o, lse, workspace});
    if (rc != FA_OK) return rc;
    int dev;
    DeviceState *st;
    rc = device_state(&dev, &st);
    if (rc != FA_OK) return rc;
    if (workspace_bytes < decode_workspace_bytes(B, H, n_q, N, D, st->num_sms)) return FA_ERR_WORKSPACE;
    DecodeArgs a{q, k, v, o, lse, static_cast<float *>(workspace), B, H, n_q, N, D, 0, 0, scale * log2e(),
                 causal ? 1 : 0};
    decode_split(B, H, n_q, N, D, st->num_sms, &a.splits, &a.chunk);
    cudaError_t e = launch_decode(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

static_assert(kDecodeScratchBytes == FA_DECODE_NOALLOC_SCRATCH_BYTES, "scratch size differs from fa.h");

// fa_decode with the partials in the library's static scratch instead of a
// caller workspace: same validation and kernels, no allocation anywhere.
extern "C" int fa_decode_noalloc(const void *q, const void *k, const void *v, void *o, float *lse, int B, int H,
                                 int n_q, int N, int D, float scale, int causal, void *stream) {
    int rc = check_decode(B, H, n_q, N, D, scale);
    if (rc != FA_OK) return rc;
    if (decode_workspace_bytes(B, H, n_q, N, D, current_num_sms()) > kDecodeScratchBytes)
        return FA_ERR_SCRATCH_LIMIT;
    rc = check_ptrs({q, k, v, o, lse});
    if (rc != FA_OK) return rc;
    int dev;
    DeviceState *st;
    rc = device_state(&dev, &st);
    if (rc != FA_OK) return rc;
    if (decode_workspace_bytes(B, H, n_q, N, D, st->num_sms) > kDecodeScratchBytes) return FA_ERR_SCRATCH_LIMIT;
    float *scratch = nullptr;
    if (decode_static_scratch(&scratch) != cudaSuccess) return FA_ERR_CUDA;
    DecodeArgs a{q, k, v, o, lse, scratch, B, H, n_q, N, D, 0, 0, scale * log2e(), causal ? 1 : 0};
    decode_split(B, H, n_q, N, D, st->num_sms, &a.splits, &a.chunk);
    cudaError_t e = launch_decode(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// ---------------------------------------------------------------- windowed and shared-prefix attention
namespace {
// Finite in units of log2 as well, and positive: the row maximum is taken before the scale.
bool scale_ok(float scale) { return scale > 0.f && std::isfinite(scale * log2e()); }

// Sizes and mask of windowed attention: 1 <= Nq <= Nk, Hq a multiple of Hkv.
int check_window(int B, int Hq, int Hkv, int Nq, int Nk, int kv_rows, int D, int window, int sinks, float scale) {
    if (B < 1 || Hq < 1 || Hkv < 1 || Nq < 1 || Nk < 1 || D < 1) return FA_ERR_SHAPE;
    if (B > 65535 || Hq > 65535 || Hq % Hkv != 0) return FA_ERR_SHAPE;
    if (Nq > Nk || kv_rows < Nk || Nk > kMaxPositions) return FA_ERR_SHAPE;
    if (window < 1 || sinks < 0) return FA_ERR_SHAPE;
    if (std::min<long long>(Nk, (long long)window + sinks) > kMaxSum) return FA_ERR_SHAPE;  // the keys that a row sees
    const long long max = (1ll << 31) - (1 << 20);  // an index, and a persistent grid's stride past it
    if ((long long)B * Hq * Nq > max || (long long)B * Hkv * kv_rows > max) return FA_ERR_SHAPE;
    if (!scale_ok(scale)) return FA_ERR_SCALE;
    if (!bf16_head_dim_ok(D)) return FA_ERR_HEAD_DIM;
    return FA_OK;
}

// The backward's: the rows of a group whose window holds a key.  (Those that see it as a sink are cut into chunks.)
int check_window_grads(int B, int Hq, int Hkv, int Nq, int Nk, int D, int window, int sinks, float scale) {
    const int rc = check_window(B, Hq, Hkv, Nq, Nk, Nk, D, window, sinks, scale);
    if (rc != FA_OK) return rc;
    return (long long)(Hq / Hkv) * std::min(Nq, window) > kMaxSum ? FA_ERR_SHAPE : FA_OK;
}

WinArgs window_args(int Hkv, int Nk, int window, int sinks) {
    WinArgs w{Hkv, Nk, std::min(window, Nk), std::min(sinks, Nk), 0, 0, 0};
    if (w.window == Nk) w.sinks = 0;  // every earlier key is in the window
    return w;
}

// Cuts the rows behind the sink tiles' windows (dK/dV) into chunks.  Without it one CTA per sink tile and key head
// meets every row: at Nq = 4096, window 1024, groups of 4 heads it took 256 of the others' 72 steps and the launch
// waited for it.
WinArgs window_args_dkdv(int B, int Hq, int Hkv, int Nq, int Nk, int D, int window, int sinks, int num_sms) {
    WinArgs w = window_args(Hkv, Nk, window, sinks);
    if (w.sinks == 0) return w;
    const long long bq = kernel_head_dim(D) == 64 ? 128 : kDkdvQRows, bk = 128, G = Hq / Hkv;
    // 64-bit sizes: tiles of rows that a key tile's window meets, rows behind the first sink tile's, and all steps
    const long long own = G * ((std::min<long long>(Nq, bk - 1 + w.window) + bq - 1) / bq);
    const long long end = std::max(0ll, std::min<long long>(Nq, bk - 1 + w.window - (Nk - Nq)));
    const long long rest = G * ((Nq - end + bq - 1) / bq);
    const long long sink_tiles = (w.sinks + bk - 1) / bk;
    const long long all = (long long)B * Hkv * ((Nk + bk - 1) / bk * own + sink_tiles * rest);
    // four sink tiles an SM balance each other uncut, and their partials would be as large as the gradients (but no sum
    // is longer than kMaxSum rows)
    const long long items = (long long)B * Hkv * sink_tiles;
    const bool fits = (own + rest) * bq <= kMaxSum;
    if (items >= 4 * num_sms && fits) return w;
    // Few sinks at D = 64: a step of a chunk costs as much as any other (1.5 us) for 16 keys or less, so win_sinks.cu takes
    // the chunks where that saves more than it costs (a launch, and Q and dO once more from HBM), unless SMs that have
    // nothing else to do would take them.  dK/dV at window 512: 32 heads of 32768 rows 464 us instead of 502, but
    // 2 x 16 (4 key heads) of 4096 rows 79 instead of 66.
    if (kernel_head_dim(D) == 64 && w.sinks <= kFewSinks) {
        const long long idle = std::max(0ll, own * num_sms - own * B * Hkv * ((Nk + bk - 1) / bk));
        const double saved_us = 1.5 * (double)(items * rest - idle) / num_sms;
        const double cost_us = 5 + (double)B * Hq * std::max(0ll, Nq - end) * D * 4 / 5.5e6;
        if (saved_us > cost_us) {
            w.few = 1;
            w.sink_tiles = 1;
            w.chunks = (int)std::max(1ll, std::min(2 * num_sms / items, rest / 4));  // one wave, two CTAs an SM
            return w;
        }
    }
    // a chunk is as long as another item, or up to four of them when that is a quarter of an SM's share of the
    // launch or less; 16 steps at least; and the launch has four chunks an SM at most beside one a sink tile
    const long long per = std::min<long long>(
        std::max({own, std::min(all / (4 * num_sms), 4 * own), 16ll, rest * items / (4 * num_sms)}), kMaxSum / bq);
    if (rest <= per / 2 && fits) return w;
    w.sink_tiles = (int)sink_tiles;
    w.chunks = (int)((rest + per - 1) / per);
    return w;
}

size_t sink_part_floats(const WinArgs &w, int B, int D) {
    return (size_t)B * w.Hkv * w.sink_tiles * (w.chunks > 0 ? 1 + w.chunks : 0) * 128 * D;
}

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// lens: null, or 4-byte aligned device memory.
int check_lens(const int *lens) {
    if (!lens) return FA_OK;
    if (!aligned4(lens)) return FA_ERR_ALIGN;
    return check_device_ptr(lens);
}

// Partials of `rows` rows: O [rows][slots][D], then (m, l) [rows][slots].
size_t partials_bytes(size_t rows, int slots, int D) { return rows * slots * ((size_t)D * 4 + 8); }
}  // namespace

extern "C" int fa_window_forward(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Hq, int Hkv,
                                 int Nq, int Nk, int kv_rows, int D, int window, int sinks, float scale, int dtype,
                                 void *stream) {
    if (dtype != FA_BF16) return FA_ERR_DTYPE;
    int rc = check_window(B, Hq, Hkv, Nq, Nk, kv_rows, D, window, sinks, scale);
    if (rc != FA_OK) return rc;
    rc = check_ptrs({q, k, v, o, lse});
    if (rc != FA_OK) return rc;
    int dev;
    DeviceState *st;
    rc = device_state(&dev, &st);
    if (rc != FA_OK) return rc;
    const WinArgs w = window_args(Hkv, Nk, window, sinks);
    SpanArgs a{};
    a.o = o;
    a.lse = lse;
    a.B = B, a.Hq = Hq, a.Hkv = Hkv, a.Nq = Nq, a.Nk = Nk, a.D = D;
    a.window = w.window, a.sinks = w.sinks;
    a.scale_log2 = scale * log2e();
    a.status = st->status_word;
    a.num_sms = st->num_sms;
    a.per_rows = FastDiv(B * Hq), a.per_seq = FastDiv(Hq), a.group = FastDiv(Hq / Hkv);
    // sink tiles read through maps that end at the last sink
    const int bn = win_fwd_keys(D), sink_rows = w.sinks > 0 ? w.sinks : Nk;
    CUtensorMap tq, tk, tv, tks, tvs, to;
    if (encode_rows(&tq, q, B * Hq, Nq, Nq, D, 128) != FA_OK ||
        encode_rows(&tk, k, B * Hkv, Nk, kv_rows, D, bn) != FA_OK ||
        encode_rows(&tv, v, B * Hkv, Nk, kv_rows, D, bn) != FA_OK ||
        encode_rows(&tks, k, B * Hkv, sink_rows, kv_rows, D, bn) != FA_OK ||
        encode_rows(&tvs, v, B * Hkv, sink_rows, kv_rows, D, bn) != FA_OK ||
        encode_rows(&to, o, B * Hq, Nq, Nq, D, 128) != FA_OK)
        return FA_ERR_CUDA;
    cudaError_t e = launch_win_fwd(a, tq, tk, tv, tks, tvs, to, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

namespace {
struct WinBackward {
    const void *q, *k, *v, *o, *dO;
    const float *lse;
    float *delta;
    void *dq, *dk, *dv;
    int B, Hq, Hkv, Nq, Nk, D, window, sinks;
    float scale;
    int grad_dtype;
    void *workspace;
    size_t workspace_bytes;
};

int check_window_backward(const WinBackward &w, int dtype) {
    if (dtype != FA_BF16 || (w.grad_dtype != FA_BF16 && w.grad_dtype != FA_F32)) return FA_ERR_DTYPE;
    return check_window_grads(w.B, w.Hq, w.Hkv, w.Nq, w.Nk, w.D, w.window, w.sinks, w.scale);
}

int window_dq(const WinBackward &w, const DeviceState &st, cudaStream_t s) {
    const int B = w.B, Hq = w.Hq, Hkv = w.Hkv, Nq = w.Nq, Nk = w.Nk, D = w.D;
    BwdArgs a{w.q, w.k, w.v, w.o, w.dO, w.lse, w.delta, w.dq, nullptr, nullptr, B, Hq, Nq, D, w.scale, w.scale * log2e(), 1,
              w.grad_dtype == FA_BF16 ? 1 : 0, st.status_word, B * Hq, window_args(Hkv, Nk, w.window, w.sinks)};
    CUtensorMap tq, tk, tv, tdo, to, tdq;
    const int k_box = kernel_head_dim(D) == 64 ? 128 : kDqKRows;
    if (encode_rows(&tq, w.q, B * Hq, Nq, Nq, D, 128) != FA_OK || encode_rows(&tk, w.k, B * Hkv, Nk, Nk, D, k_box) != FA_OK ||
        encode_rows(&tv, w.v, B * Hkv, Nk, Nk, D, k_box) != FA_OK ||
        encode_rows(&tdo, w.dO, B * Hq, Nq, Nq, D, 128) != FA_OK || encode_rows(&to, w.o, B * Hq, Nq, Nq, D, 128) != FA_OK ||
        encode_3d(&tdq, w.dq, B * Hq, Nq, D, 128, w.grad_dtype == FA_F32) != FA_OK)
        return FA_ERR_CUDA;
    const bool early = Nk - Nq < kExactDelta;
    cudaError_t e = early ? launch_win_delta(a, s) : cudaSuccess;
    if (e == cudaSuccess) e = launch_win_dq(a, tq, tk, tv, tdo, to, tdq, st.num_sms, early, s);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// The sink tiles' partials of dK, then of dV, in the workspace; checks that it holds them.
int check_window_workspace(const WinBackward &w, const WinArgs &win) {
    const size_t floats = sink_part_floats(win, w.B, w.D);
    if (floats == 0) return FA_OK;
    const int rc = check_ptrs({w.workspace});
    if (rc != FA_OK) return rc;
    return w.workspace_bytes < 2 * floats * sizeof(float) ? FA_ERR_WORKSPACE : FA_OK;
}

int window_dkdv(const WinBackward &w, const WinArgs &win, const DeviceState &st, bool behind, cudaStream_t s) {
    const int B = w.B, Hq = w.Hq, Hkv = w.Hkv, Nq = w.Nq, Nk = w.Nk, D = w.D;
    BwdArgs a{w.q, w.k, w.v, nullptr, w.dO, w.lse, w.delta, nullptr, w.dk, w.dv, B, Hq, Nq, D, w.scale, w.scale * log2e(), 1,
              w.grad_dtype == FA_BF16 ? 1 : 0, st.status_word, B * Hkv, win};
    const size_t part_floats = sink_part_floats(win, B, D);
    float *part_dk = static_cast<float *>(w.workspace), *part_dv = part_dk + part_floats;
    CUtensorMap tq, tk, tv, tdo, tdk, tdv, parts[2];
    const int q_box = kernel_head_dim(D) == 64 ? 128 : kDkdvQRows;
    const bool f32 = w.grad_dtype == FA_F32;
    if (encode_rows(&tq, w.q, B * Hq, Nq, Nq, D, q_box) != FA_OK || encode_rows(&tk, w.k, B * Hkv, Nk, Nk, D, 128) != FA_OK ||
        encode_rows(&tv, w.v, B * Hkv, Nk, Nk, D, 128) != FA_OK ||
        encode_rows(&tdo, w.dO, B * Hq, Nq, Nq, D, q_box) != FA_OK ||
        encode_3d(&tdk, w.dk, B * Hkv, Nk, D, 128, f32) != FA_OK || encode_3d(&tdv, w.dv, B * Hkv, Nk, D, 128, f32) != FA_OK)
        return FA_ERR_CUDA;
    parts[0] = tdk, parts[1] = tdv;
    if (part_floats > 0) {
        const int n = B * Hkv * win.sink_tiles * (1 + win.chunks);
        if (encode_3d(&parts[0], part_dk, n, 128, D, 128, true) != FA_OK ||
            encode_3d(&parts[1], part_dv, n, 128, D, 128, true) != FA_OK)
            return FA_ERR_CUDA;
    }
    cudaError_t e = launch_win_dkdv(a, tq, tk, tv, tdo, tdk, tdv, parts, st.num_sms, behind, s);
    if (e == cudaSuccess && win.few) e = launch_win_sinks(a, tq, tdo, part_dk, part_dv, s);
    if (e == cudaSuccess && part_floats > 0) e = launch_sink_sum(a, part_dk, part_dv, s);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
}  // namespace

extern "C" int fa_window_backward_dq(const void *q, const void *k, const void *v, const void *o, const void *dO,
                                     const float *lse, float *delta, void *dq, int B, int Hq, int Hkv, int Nq, int Nk,
                                     int D, int window, int sinks, float scale, int dtype, int grad_dtype,
                                     void *stream) {
    const WinBackward w{q, k, v, o, dO, lse, delta, dq, nullptr, nullptr, B, Hq, Hkv, Nq, Nk, D, window, sinks, scale,
                        grad_dtype, nullptr, 0};
    int rc = check_window_backward(w, dtype);
    if (rc != FA_OK) return rc;
    rc = check_ptrs({q, k, v, o, dO, lse, delta, dq});
    if (rc != FA_OK) return rc;
    int dev;
    DeviceState *st;
    rc = device_state(&dev, &st);
    if (rc != FA_OK) return rc;
    return window_dq(w, *st, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int fa_window_backward_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Nk, int D, int window, int sinks,
                                                  size_t *bytes) {
    if (!bytes) return FA_ERR_NULL;
    int rc = check_window_grads(B, Hq, Hkv, Nq, Nk, D, window, sinks, 1.f);
    if (rc != FA_OK) return rc;
    *bytes = 2 * sizeof(float) *
             sink_part_floats(window_args_dkdv(B, Hq, Hkv, Nq, Nk, D, window, sinks, current_num_sms()), B, D);
    return FA_OK;
}

extern "C" int fa_window_backward_dkdv(const void *q, const void *k, const void *v, const void *dO, const float *lse,
                                       const float *delta, void *dk, void *dv, int B, int Hq, int Hkv, int Nq, int Nk,
                                       int D, int window, int sinks, float scale, int dtype, int grad_dtype,
                                       void *workspace, size_t workspace_bytes, void *stream) {
    const WinBackward w{q, k, v, nullptr, dO, lse, const_cast<float *>(delta), nullptr, dk, dv, B, Hq, Hkv, Nq, Nk, D, window,
                        sinks, scale, grad_dtype, workspace, workspace_bytes};
    int rc = check_window_backward(w, dtype);
    if (rc != FA_OK) return rc;
    rc = check_ptrs({q, k, v, dO, lse, delta, dk, dv});
    if (rc != FA_OK) return rc;
    int dev;
    DeviceState *st;
    rc = device_state(&dev, &st);
    if (rc != FA_OK) return rc;
    const WinArgs win = window_args_dkdv(B, Hq, Hkv, Nq, Nk, D, window, sinks, st->num_sms);
    rc = check_window_workspace(w, win);
    if (rc != FA_OK) return rc;
    return window_dkdv(w, win, *st, false, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int fa_window_backward(const void *q, const void *k, const void *v, const void *o, const void *dO,
                                  const float *lse, float *delta, void *dq, void *dk, void *dv, int B, int Hq, int Hkv,
                                  int Nq, int Nk, int D, int window, int sinks, float scale, int dtype, int grad_dtype,
                                  void *workspace, size_t workspace_bytes, void *stream) {
    const WinBackward w{q, k, v, o, dO, lse, delta, dq, dk, dv, B, Hq, Hkv, Nq, Nk, D, window, sinks, scale, grad_dtype,
                        workspace, workspace_bytes};
    int rc = check_window_backward(w, dtype);
    if (rc != FA_OK) return rc;
    rc = check_ptrs({q, k, v, o, dO, lse, delta, dq, dk, dv});
    if (rc != FA_OK) return rc;
    int dev;
    DeviceState *st;
    rc = device_state(&dev, &st);
    if (rc != FA_OK) return rc;
    const WinArgs win = window_args_dkdv(B, Hq, Hkv, Nq, Nk, D, window, sinks, st->num_sms);
    rc = check_window_workspace(w, win);
    if (rc != FA_OK) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    rc = window_dq(w, *st, s);
    return rc != FA_OK ? rc : window_dkdv(w, win, *st, true, s);
}

namespace {
constexpr int kMaxDecodeRows = 16;  // new rows per sequence

int check_rows(int B, int Hq, int Hkv, int n_q, int N, int D, float scale) {
    if (B < 1 || Hq < 1 || Hkv < 1 || n_q < 1 || N < 1 || D < 1) return FA_ERR_SHAPE;
    if (B > 65535 || Hq > 65535 || Hq % Hkv != 0 || n_q > kMaxDecodeRows || N > kMaxPositions) return FA_ERR_SHAPE;
    const long long max = (1ll << 31) - (1 << 20);
    if ((long long)B * Hkv * N > max || (long long)B * Hq * n_q > max) return FA_ERR_SHAPE;
    if (!scale_ok(scale)) return FA_ERR_SCALE;
    if (D != 64 && D != 128 && D != 256) return FA_ERR_HEAD_DIM;
    return FA_OK;
}

// CTAs per (sequence, key head, row tile) of windowed decode, and whether they join their rows as a cluster.
struct TokenPlan {
    int splits, cluster;
};
TokenPlan token_plan(int B, int Hq, int Hkv, int n_q, int N, int D, const WinArgs &w, int num_sms) {
    // the most key tiles any sequence can need: a cache full of keys, or the window of the n_q rows and the sinks
    const int bn = win_decode_tile_keys();
    const KeySpan sp = key_span(std::max(0, N - n_q), N - 1, w.window, w.sinks, bn);
    const int splits = win_decode_splits(B, Hkv, Hq / Hkv * n_q, sp.n, D, num_sms);
    const int cluster = win_decode_cluster(splits, sp.n);
    return TokenPlan{cluster > 0 ? cluster : splits, cluster > 0 ? 1 : 0};
}

size_t token_workspace(int B, int Hq, int n_q, int D, const TokenPlan &p) {
    return p.splits > 1 && !p.cluster ? partials_bytes((size_t)B * Hq * n_q, p.splits, D) : 0;
}

int check_token(int B, int Hq, int Hkv, int n_q, int N, int D, int window, int sinks, float scale) {
    int rc = check_rows(B, Hq, Hkv, n_q, N, D, scale);
    if (rc == FA_OK && (window < 1 || sinks < 0 || n_q > N)) rc = FA_ERR_SHAPE;
    return rc;
}
}  // namespace

extern "C" int fa_window_decode_workspace_bytes(int B, int Hq, int Hkv, int n_q, int N, int D, int window, int sinks,
                                                size_t *bytes) {
    if (!bytes) return FA_ERR_NULL;
    int rc = check_token(B, Hq, Hkv, n_q, N, D, window, sinks, 1.f);
    if (rc != FA_OK) return rc;
    const WinArgs w = window_args(Hkv, N, window, sinks);
    *bytes = token_workspace(B, Hq, n_q, D, token_plan(B, Hq, Hkv, n_q, N, D, w, current_num_sms()));
    return FA_OK;
}

extern "C" int fa_window_decode(const void *q, const void *k, const void *v, const int *lens, void *o, float *lse, int B,
                                int Hq, int Hkv, int n_q, int N, int D, int window, int sinks, float scale,
                                void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_token(B, Hq, Hkv, n_q, N, D, window, sinks, scale);
    if (rc != FA_OK) return rc;
    rc = check_ptrs({q, k, v, o, lse});
    if (rc != FA_OK) return rc;
    rc = check_lens(lens);
    if (rc != FA_OK) return rc;
    int dev;
    DeviceState *st;
    rc = device_state(&dev, &st);
    if (rc != FA_OK) return rc;
    const WinArgs w = window_args(Hkv, N, window, sinks);
    const TokenPlan plan = token_plan(B, Hq, Hkv, n_q, N, D, w, st->num_sms);
    const size_t need = token_workspace(B, Hq, n_q, D, plan);
    if (need > 0) {
        rc = check_ptrs({workspace});
        if (rc != FA_OK) return rc;
        if (workspace_bytes < need) return FA_ERR_WORKSPACE;
    }
    const size_t rows = (size_t)B * Hq * n_q;
    float *part_o = need > 0 ? static_cast<float *>(workspace) : nullptr;
    float2 *part_ml = need > 0 ? reinterpret_cast<float2 *>(part_o + rows * plan.splits * D) : nullptr;
    const WinDecodeArgs a{q, lens, o, lse, B, Hkv, Hq / Hkv * n_q, n_q, N, D, w.window, w.sinks, scale * log2e(),
                          st->status_word, plan.splits, part_o, part_ml, plan.cluster, part_o == nullptr, PrefixParts{}, 0};
    CUtensorMap tk, tv;
    if (encode_rows(&tk, k, B * Hkv, N, N, D, win_decode_tile_keys()) != FA_OK ||
        encode_rows(&tv, v, B * Hkv, N, N, D, win_decode_tile_keys()) != FA_OK)
        return FA_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = launch_win_decode(a, tk, tv, s);
    if (e == cudaSuccess && part_o) e = launch_win_join(a, PrefixParts{}, s);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

namespace {
// How shared-prefix decode cuts its work: the prefix into chunks for packed 128-row query tiles on `ctas` SMs, the
// sequences' own caches into `own` CTAs each, which run on the other SMs meanwhile and on all of them afterwards.
struct PrefixPlan {
    int R, rb, nb, m_tiles, splits, chunk_tiles, own, ctas;
    bool fused;  // both fit on the GPU at once: the own caches' CTAs join the prefix's partials
    // 128-row partials of the prefix, and partials of the own caches' rows
    size_t prefix_parts(int Hkv) const { return (size_t)Hkv * m_tiles * splits; }
    size_t own_parts(size_t rows) const { return fused ? 0 : rows * own; }
    size_t bytes(int Hkv, size_t rows, int D) const {
        return (prefix_parts(Hkv) * 128 + own_parts(rows)) * ((size_t)D * 4 + 8);
    }
};

PrefixPlan prefix_plan(int B, int Hq, int Hkv, int n_q, int P, int N, int D, int num_sms) {
    PrefixPlan p;
    p.R = Hq / Hkv * n_q;
    p.rb = std::min(p.R, 128);
    p.nb = std::min(128 / p.rb, B);
    p.m_tiles = p.R <= 128 ? (B + p.nb - 1) / p.nb : B * ((p.R + 127) / 128);
    const int Dk = kernel_head_dim(D), bn = fwd_block_n(Dk), tiles = (P + bn - 1) / bn;
    const int per_block = Dk <= 128 ? 2 : 1;  // query tiles a block streams the chunk past
    const int units = Hkv * ((p.m_tiles + per_block - 1) / per_block);
    p.own = win_decode_splits(B, Hkv, p.R, (N + win_decode_tile_keys() - 1) / win_decode_tile_keys(), D, num_sms);
    const int own_sms = win_decode_sms(B, Hkv, p.R, p.own, D);
    p.fused = p.own == 1 && own_sms + std::min(units, num_sms) <= num_sms;
    // Measured: a key tile takes a block about 1.4 us (D = 64), 1.7 (128), 1.0 (256, 64 keys), a block 3 tiles' time
    // besides; an SM on its own streams about 80 KB/us of caches, all of them 6500.  Half of N is taken for the length.
    const double tile_us = Dk == 64 ? 1.4 : Dk == 128 ? 1.7 : 1.0;
    const double own_kb = (double)B * Hkv * N * D * 2 / 1000;
    double best = 1e300;
    const int most = std::min(tiles, kMaxSum / bn), least = (tiles + most - 1) / most;  // a chunk's sums stay within kMaxSum
    for (int left = 0; left <= num_sms / 3; left += 8) {
        const int ctas = p.fused ? num_sms - own_sms : num_sms - left;
        for (int c = most; c >= 1; --c) {  // s chunks of c tiles, each s that a chunk size gives once, with the smallest
            const int s = (tiles + c - 1) / c;
            c = (tiles + s - 1) / s;
            if (s > least && (long long)units * s > 4ll * ctas) break;
            const double prefix_us = (double)(((long long)units * s + ctas - 1) / ctas) * (c + 3) * tile_us;
            const double rest = own_kb - std::min(own_kb, left * 80.0 * prefix_us);
            const double us = p.fused ? prefix_us : prefix_us + rest / 6500;
            if (us < best) {
                best = us;
                p.splits = s;
                p.chunk_tiles = c;
                p.ctas = ctas;
            }
            c = std::min(c, (tiles + s) / (s + 1) + 1);  // on to s + 1 chunks
        }
        if (p.fused) break;
    }
    return p;
}

// The prefix kernels store their partials 32 bytes at a time, and a caller's workspace is 16-byte aligned: the partials
// begin at its first 32-byte boundary, and the size query has room for that.
constexpr size_t kPartAlign = 32;
size_t part_shift(const void *workspace) { return -reinterpret_cast<uintptr_t>(workspace) & (kPartAlign - 1); }

int check_prefix(int B, int Hq, int Hkv, int n_q, int P, int N, int D, float scale) {
    int rc = check_rows(B, Hq, Hkv, n_q, N, D, scale);
    if (rc == FA_OK && (P < 1 || P > kMaxPositions || (long long)Hkv * P > (1ll << 31) - 1)) rc = FA_ERR_SHAPE;
    return rc;
}
}  // namespace

extern "C" int fa_prefix_decode_workspace_bytes(int B, int Hq, int Hkv, int n_q, int P, int N, int D, size_t *bytes) {
    if (!bytes) return FA_ERR_NULL;
    int rc = check_prefix(B, Hq, Hkv, n_q, P, N, D, 1.f);
    if (rc != FA_OK) return rc;
    const PrefixPlan p = prefix_plan(B, Hq, Hkv, n_q, P, N, D, current_num_sms());
    *bytes = p.bytes(Hkv, (size_t)B * Hq * n_q, D) + kPartAlign - 16;
    return FA_OK;
}

extern "C" int fa_prefix_decode(const void *q, const void *k_prefix, const void *v_prefix, const void *k, const void *v,
                                const int *lens, void *o, float *lse, int B, int Hq, int Hkv, int n_q, int P, int N,
                                int D, float scale, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_prefix(B, Hq, Hkv, n_q, P, N, D, scale);
    if (rc != FA_OK) return rc;
    rc = check_ptrs({q, k_prefix, v_prefix, k, v, o, lse, workspace});
    if (rc != FA_OK) return rc;
    rc = check_lens(lens);
    if (rc != FA_OK) return rc;
    int dev;
    DeviceState *st;
    rc = device_state(&dev, &st);
    if (rc != FA_OK) return rc;
    const PrefixPlan p = prefix_plan(B, Hq, Hkv, n_q, P, N, D, st->num_sms);
    const size_t rows = (size_t)B * Hq * n_q;
    const size_t shift = part_shift(workspace);
    if (workspace_bytes < shift + p.bytes(Hkv, rows, D)) return FA_ERR_WORKSPACE;
    // O of the prefix's partials and of the rows' own, then (m, l) of both
    PrefixParts parts{reinterpret_cast<float *>(static_cast<char *>(workspace) + shift), nullptr, p.m_tiles, p.splits, p.R, p.rb, p.nb};
    float *own_o = parts.o + p.prefix_parts(Hkv) * 128 * D;
    parts.ml = reinterpret_cast<float2 *>(own_o + p.own_parts(rows) * D);
    float2 *own_ml = parts.ml + p.prefix_parts(Hkv) * 128;

    SpanArgs a{};
    a.B = B, a.Hq = Hq, a.Hkv = Hkv, a.Nq = n_q, a.Nk = P, a.D = D;
    a.window = P;
    a.scale_log2 = scale * log2e();
    a.status = st->status_word;
    a.num_sms = p.ctas;
    a.parts = parts;
    a.chunk_tiles = p.chunk_tiles;
    // the rows of a key head: [B, Hkv, R, D], boxes of rb rows of nb sequences
    CUtensorMap tq, tkp, tvp, tk, tv;
    {
        cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)p.R, (cuuint64_t)Hkv, (cuuint64_t)B};
        cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)p.R * D * 2, (cuuint64_t)Hkv * p.R * D * 2};
        cuuint32_t box[4] = {64, (cuuint32_t)p.rb, 1, (cuuint32_t)p.nb};
        cuuint32_t estr[4] = {1, 1, 1, 1};
        if (g_encode(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(q), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return FA_ERR_CUDA;
    }
    const int bn = fwd_block_n(kernel_head_dim(D)), own_box = win_decode_tile_keys();
    if (encode_rows(&tkp, k_prefix, Hkv, P, P, D, bn) != FA_OK || encode_rows(&tvp, v_prefix, Hkv, P, P, D, bn) != FA_OK ||
        encode_rows(&tk, k, B * Hkv, N, N, D, own_box) != FA_OK || encode_rows(&tv, v, B * Hkv, N, N, D, own_box) != FA_OK)
        return FA_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = launch_win_fwd(a, tq, tkp, tvp, tkp, tvp, tkp, s);
    if (e != cudaSuccess) return FA_ERR_CUDA;
    const WinDecodeArgs d{q, lens, o, lse, B, Hkv, p.R, n_q, N, D, N, 0, scale * log2e(), st->status_word, p.own,
                          own_o, own_ml, 0, p.fused, parts, 1};
    e = launch_win_decode(d, tk, tv, s);
    if (e == cudaSuccess && !p.fused) e = launch_win_join(d, parts, s);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

extern "C" const char *fa_status_string(int status) {
    switch (status) {
        case FA_OK: return "ok";
        case FA_ERR_NULL: return "a required pointer is NULL";
        case FA_ERR_SHAPE: return "invalid shape (sizes must be >= 1, within index limits and fit together)";
        case FA_ERR_HEAD_DIM: return "head dimension not supported for this dtype / pass";
        case FA_ERR_DTYPE: return "unsupported dtype or grad_dtype";
        case FA_ERR_ALIGN: return "pointer not 16-byte aligned";
        case FA_ERR_SCALE: return "scale is not finite, or not positive where it has to be";
        case FA_ERR_CUDA: return "CUDA runtime error";
        case FA_ERR_TIMEOUT: return "a bounded in-kernel wait ran out";
        case FA_ERR_DEVICE_PTR: return "pointer is not device-accessible memory";
        case FA_ERR_DEVICE: return "current device is not sm_103 (GB300)";
        case FA_ERR_WORKSPACE: return "workspace smaller than its size query requires";
        case FA_ERR_SCRATCH_LIMIT:
            return "sizes need more than FA_DECODE_NOALLOC_SCRATCH_BYTES of scratch; use fa_decode with a workspace";
        default: return "unknown status";
    }
}

extern "C" int fa_device_status(void *stream) {
    int dev;
    DeviceState *st;
    int rc = device_state(&dev, &st);
    if (rc != FA_OK) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(s) != cudaSuccess) return FA_ERR_CUDA;
    int word = 0, zero = 0;
    if (cudaMemcpy(&word, st->status_word, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return FA_ERR_CUDA;
    if (word != 0 && cudaMemcpy(st->status_word, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess)
        return FA_ERR_CUDA;
    if (word == 0) return FA_OK;
    return -(word & 0xFFFF);
}

namespace fa {
namespace {
// One warp waits on a barrier that nothing arrives on; the wait is bounded
// and records FA_ERR_TIMEOUT when it runs out.
__global__ void selftest_timeout_kernel(int *status, unsigned long long limit_ns) {
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_mbarrier_init();
    }
    __syncthreads();
    if (threadIdx.x == 0) mbar_wait(&bar, 0, status, 99, limit_ns);
    __syncthreads();
}
}  // namespace

cudaError_t launch_selftest_timeout(int *status, int limit_us, cudaStream_t s) {
    selftest_timeout_kernel<<<1, 32, 0, s>>>(status, (unsigned long long)limit_us * 1000ull);
    return cudaGetLastError();
}
}  // namespace fa

extern "C" int fa_selftest_timeout(int limit_us, void *stream) {
    if (limit_us < 1 || limit_us > 2000000) return FA_ERR_SHAPE;
    int dev;
    DeviceState *st;
    int rc = device_state(&dev, &st);
    if (rc != FA_OK) return rc;
    cudaError_t e = launch_selftest_timeout(st->status_word, limit_us, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

namespace fa {
namespace {
__global__ void selftest_exp2_kernel(const float *x, float *y, int n) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) y[i] = ex2_fma(x[i]);
}
}  // namespace
}  // namespace fa

extern "C" int fa_selftest_exp2(const float *x, float *y, int n, void *stream) {
    if (n < 1) return FA_ERR_SHAPE;
    int rc = check_ptrs({x, y});
    if (rc != FA_OK) return rc;
    int dev;
    DeviceState *st;
    rc = device_state(&dev, &st);
    if (rc != FA_OK) return rc;
    selftest_exp2_kernel<<<(n + 255) / 256, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(x, y, n);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

extern "C" int fa_version(void) { return 100; }
