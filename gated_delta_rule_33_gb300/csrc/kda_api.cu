// kda_api.cu -- the extern "C" entry points of libkda (declared in include/kda.h).
//
// Host-side argument checks, the per-device error word, and the launches.  No
// CUDA allocation happens here; every buffer is the caller's.
#include <mutex>
#include <vector>

#include "../../include/kda.h"
#include "kda_internal.cuh"
#include "kda_paged.cuh"
#include "kda_tree.cuh"

namespace {

// One error word per device: kernels record the first error they meet, the
// host reads and clears it in kda_get_last_device_error().
__device__ unsigned int g_device_error_word;

constexpr int kMaxDevices = 64;
struct DeviceInfo {
    bool ready = false;
    bool supported = false;
    int num_sms = 0;
    unsigned int *error_word = nullptr;
};
DeviceInfo g_devices[kMaxDevices];
std::mutex g_devices_mutex;

// Looks up (once per device) the SM count, whether the device is an sm_103
// part this library was built for, and the device address of the error word.
kda_status current_device(DeviceInfo **out) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return KDA_ERR_NO_DEVICE;
    }
    std::lock_guard<std::mutex> lock(g_devices_mutex);
    DeviceInfo &info = g_devices[dev];
    if (!info.ready) {
        cudaDeviceProp prop;
        if (cudaGetDeviceProperties(&prop, dev) != cudaSuccess) {
            cudaGetLastError();
            return KDA_ERR_NO_DEVICE;
        }
        info.supported = (prop.major == 10 && prop.minor == 3);
        info.num_sms = prop.multiProcessorCount;
        void *addr = nullptr;
        if (cudaGetSymbolAddress(&addr, g_device_error_word) != cudaSuccess) {
            cudaGetLastError();
            return KDA_ERR_CUDA;
        }
        info.error_word = static_cast<unsigned int *>(addr);
        info.ready = true;
    }
    if (!info.supported) return KDA_ERR_NO_DEVICE;
    *out = &info;
    return KDA_OK;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool valid_dtype(kda_dtype d) { return d == KDA_BF16 || d == KDA_FP32; }

// Whether two byte ranges share an address.
inline bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    return a != nullptr && b != nullptr && na > 0 && nb > 0 && pa < pb + nb && pb < pa + na;
}

struct Buffer {
    const void *p;
    size_t bytes;
};

// Whether [a, a + na) meets one of n rows of `row` bytes, `stride` bytes (not below `row`) apart.
inline bool overlaps_rows(const void *a, size_t na, const void *b, size_t row, size_t stride, int64_t n) {
    if (n <= 1) return n == 1 && overlaps(a, na, b, row);
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    if (a == nullptr || b == nullptr || na == 0 || row == 0) return false;
    // the first row that ends behind a's begin
    const size_t first = pa < pb + row ? 0 : (pa - pb - row) / stride + 1;
    return first < static_cast<size_t>(n) && pb + first * stride < pa + na;
}

kda_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return KDA_OK;
    cudaGetLastError();
    return KDA_ERR_CUDA;
}

// Host checks of kda_chunk_prefill's arguments other than the workspace.
kda_status check_prefill_args(const void *q, const void *k, const void *v, const float *g,
                              const float *beta, const int32_t *cu_seqlens, int B, int64_t N,
                              int H, int K, int V, const float *initial_state,
                              const float *final_state, const void *o, kda_dtype o_dtype) {
    if (N < 0 || B < 1 || H < 1) return KDA_ERR_INVALID_ARG;
    if (K != 128 || V != 128) return KDA_ERR_UNSUPPORTED_SHAPE;
    if (!valid_dtype(o_dtype)) return KDA_ERR_UNSUPPORTED_DTYPE;
    if (cu_seqlens == nullptr && B != 1) return KDA_ERR_INVALID_ARG;
    if (N > 0 && (q == nullptr || k == nullptr || v == nullptr || g == nullptr ||
                  beta == nullptr || o == nullptr))
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(beta) ||
        !aligned16(o) || !aligned16(initial_state) || !aligned16(final_state) ||
        !aligned16(cu_seqlens))
        return KDA_ERR_MISALIGNED;
    return KDA_OK;
}

// Checks a cache description and turns it into what the kernels take.
kda_status paged_view(const kda_paged_cache *c, kda::PagedView *view) {
    if (c == nullptr || c->num_pages < 1 || c->page_size < 1 || c->heads < 1)
        return KDA_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
        return KDA_ERR_UNSUPPORTED_SHAPE;
    if (c->dtype != KDA_BF16 && c->dtype != KDA_FP8_E4M3) return KDA_ERR_UNSUPPORTED_DTYPE;
    if (static_cast<int64_t>(c->num_pages) * c->page_size > INT32_MAX ||
        static_cast<int64_t>(c->heads) * c->head_dim > INT32_MAX / 4)
        return KDA_ERR_UNSUPPORTED_SHAPE;
    if (c->k == nullptr || c->v == nullptr) return KDA_ERR_INVALID_ARG;
    if ((c->k_scale == nullptr) != (c->v_scale == nullptr)) return KDA_ERR_INVALID_ARG;
    const bool fp8 = c->dtype == KDA_FP8_E4M3;
    if (!fp8 && c->k_scale != nullptr) return KDA_ERR_INVALID_ARG;
    const int64_t size = fp8 ? 1 : 2;
    // The rows of head_dim values must not overlap: in order of their strides,
    // each dimension of more than one entry steps past all that lies inside it.
    struct Dim {
        int64_t stride, count;
    } d[3] = {{c->head_stride, c->heads},
              {c->token_stride, c->page_size},
              {c->page_stride, c->num_pages}};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (d[j].stride > d[j + 1].stride) {
                const Dim x = d[j];
                d[j] = d[j + 1];
                d[j + 1] = x;
            }
    int64_t inside = c->head_dim;
    for (const Dim &x : d) {
        if (x.count == 1) continue;
        if (x.stride < inside) return KDA_ERR_INVALID_ARG;
        if (x.stride > INT64_MAX / 8 / x.count) return KDA_ERR_INVALID_ARG;
        if (x.stride * size % 16 != 0) return KDA_ERR_MISALIGNED;
        inside += x.stride * (x.count - 1);
    }
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale))
        return KDA_ERR_MISALIGNED;
    view->k = static_cast<uint8_t *>(c->k);
    view->v = static_cast<uint8_t *>(c->v);
    view->k_scale = c->k_scale;
    view->v_scale = c->v_scale;
    // the stride of a single entry is never taken
    view->page_stride = c->num_pages == 1 ? 0 : c->page_stride * size;
    view->token_stride = c->page_size == 1 ? 0 : c->token_stride * size;
    view->head_stride = c->heads == 1 ? 0 : c->head_stride * size;
    view->page = kda::FastDiv(static_cast<uint32_t>(c->page_size));
    view->num_pages = c->num_pages;
    view->heads = c->heads;
    view->head_dim = c->head_dim;
    view->fp8 = fp8;
    return KDA_OK;
}

// Whether kda_paged_decode takes so many query heads and sequences.
bool paged_decode_sizes(int B, int q_heads, int kv_heads, int head_dim) {
    return q_heads % kv_heads == 0 && static_cast<int64_t>(q_heads) * head_dim <= INT32_MAX &&
           static_cast<int64_t>(kv_heads) * head_dim <= INT32_MAX / 4 &&
           static_cast<int64_t>(B) * q_heads <= INT32_MAX;
}

constexpr int kMaxTreeRequests = 65535;  // a dimension of the grid

// What the calls over trees of drafted tokens have in common.
kda_status tree_sizes(int B, int64_t N, int max_nodes, int num_slots, const int32_t *slots) {
    if (B < 0 || B > kMaxTreeRequests || N < 0 || N > INT32_MAX || num_slots < 0)
        return KDA_ERR_INVALID_ARG;
    if (max_nodes < 1 || max_nodes > KDA_TREE_MAX_NODES) return KDA_ERR_UNSUPPORTED_SHAPE;
    if (slots == nullptr && num_slots < B) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

// Whether kda_paged_tree_decode takes so many query heads and nodes.
bool paged_tree_sizes(int B, int max_nodes, int q_heads, int kv_heads, int head_dim) {
    return paged_decode_sizes(B, q_heads, kv_heads, head_dim) &&
           static_cast<int64_t>(B) * q_heads <= INT32_MAX / max_nodes;
}

}  // namespace

namespace kda {

cudaError_t ensure_dynamic_smem(const void *func, int bytes) {
    struct Done {
        int dev;
        const void *func;
        int bytes;
    };
    static std::mutex m;
    static std::vector<Done> done;
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(m);
    for (const Done &d : done)
        if (d.dev == dev && d.func == func && d.bytes >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.push_back(Done{dev, func, bytes});
    return e;
}

}  // namespace kda

extern "C" {

int kda_version(void) { return KDA_VERSION; }

const char *kda_status_string(kda_status status) {
    switch (status) {
        case KDA_OK: return "KDA_OK";
        case KDA_ERR_INVALID_ARG: return "KDA_ERR_INVALID_ARG";
        case KDA_ERR_UNSUPPORTED_SHAPE: return "KDA_ERR_UNSUPPORTED_SHAPE";
        case KDA_ERR_UNSUPPORTED_DTYPE: return "KDA_ERR_UNSUPPORTED_DTYPE";
        case KDA_ERR_MISALIGNED: return "KDA_ERR_MISALIGNED";
        case KDA_ERR_WORKSPACE_TOO_SMALL: return "KDA_ERR_WORKSPACE_TOO_SMALL";
        case KDA_ERR_CUDA: return "KDA_ERR_CUDA";
        case KDA_ERR_DEVICE_TIMEOUT: return "KDA_ERR_DEVICE_TIMEOUT";
        case KDA_ERR_NONFINITE: return "KDA_ERR_NONFINITE";
        case KDA_ERR_NOT_IMPLEMENTED: return "KDA_ERR_NOT_IMPLEMENTED";
        case KDA_ERR_NO_DEVICE: return "KDA_ERR_NO_DEVICE";
        case KDA_ERR_DECAY_RANGE: return "KDA_ERR_DECAY_RANGE";
    }
    return "KDA_ERR_UNKNOWN";
}

kda_status kda_gate_fused(const void *f, kda_dtype f_dtype, const void *b, kda_dtype b_dtype,
                          const float *A_log, kda_alog_mode alog_mode, const float *dt_bias,
                          float *g_out, float *beta_out, int64_t N, int H, int K, void *stream) {
    if (N < 0 || H < 1 || K < 1) return KDA_ERR_INVALID_ARG;
    if (!valid_dtype(f_dtype) || !valid_dtype(b_dtype)) return KDA_ERR_UNSUPPORTED_DTYPE;
    if (alog_mode != KDA_ALOG_PER_HEAD && alog_mode != KDA_ALOG_PER_CHANNEL &&
        alog_mode != KDA_ALOG_PER_HEAD_CHANNEL)
        return KDA_ERR_INVALID_ARG;
    if ((b == nullptr) != (beta_out == nullptr)) return KDA_ERR_INVALID_ARG;
    if (N > 0 && (f == nullptr || g_out == nullptr)) return KDA_ERR_INVALID_ARG;
    if (A_log == nullptr || dt_bias == nullptr) return KDA_ERR_INVALID_ARG;
    if (!aligned16(f) || !aligned16(b) || !aligned16(A_log) || !aligned16(dt_bias) ||
        !aligned16(g_out) || !aligned16(beta_out))
        return KDA_ERR_MISALIGNED;
    if (N == 0) return KDA_OK;
    DeviceInfo *dev = nullptr;
    kda_status st = current_device(&dev);
    if (st != KDA_OK) return st;
    return from_cuda(kda::launch_gate(f, f_dtype == KDA_BF16, b, b_dtype == KDA_BF16, A_log,
                                      static_cast<int>(alog_mode), dt_bias, g_out, beta_out, N, H,
                                      K, dev->num_sms, static_cast<cudaStream_t>(stream)));
}

size_t kda_chunk_prefill_workspace_size(int64_t N, int B, int H, int K, int V) {
    if (N < 0 || B < 1 || H < 1 || K != 128 || V != 128) return 0;
    return kda::prefill_workspace_bytes(N, B, H);
}

kda_status kda_chunk_prefill(const void *q, const void *k, const void *v, const float *g,
                             const float *beta, const int32_t *cu_seqlens, int B, int64_t N, int H,
                             int K, int V, float scale, const float *initial_state,
                             float *final_state, void *o, kda_dtype o_dtype, void *workspace,
                             size_t workspace_bytes, void *stream) {
    kda_status st = check_prefill_args(q, k, v, g, beta, cu_seqlens, B, N, H, K, V, initial_state,
                                       final_state, o, o_dtype);
    if (st != KDA_OK) return st;
    if (!aligned16(workspace)) return KDA_ERR_MISALIGNED;
    const size_t need = kda::prefill_workspace_bytes(N, B, H);
    if (workspace_bytes < need || (need > 0 && workspace == nullptr))
        return KDA_ERR_WORKSPACE_TOO_SMALL;
    DeviceInfo *dev = nullptr;
    st = current_device(&dev);
    if (st != KDA_OK) return st;
    return from_cuda(kda::launch_prefill(
        static_cast<const __nv_bfloat16 *>(q), static_cast<const __nv_bfloat16 *>(k),
        static_cast<const __nv_bfloat16 *>(v), g, beta, cu_seqlens, B, N, H, scale, initial_state,
        final_state, o, o_dtype == KDA_BF16, workspace, dev->error_word, dev->num_sms,
        static_cast<cudaStream_t>(stream)));
}

kda_status kda_chunk_prefill_gated(const void *q, const void *k, const void *v, const void *f,
                                   kda_dtype f_dtype, const void *b, kda_dtype b_dtype,
                                   const float *A_log, kda_alog_mode alog_mode,
                                   const float *dt_bias, const int32_t *cu_seqlens, int B,
                                   int64_t N, int H, int K, int V, float scale,
                                   const float *initial_state, float *final_state, void *o,
                                   kda_dtype o_dtype, void *workspace, size_t workspace_bytes,
                                   void *stream) {
    if (N < 0 || B < 1 || H < 1) return KDA_ERR_INVALID_ARG;
    if (K != 128 || V != 128) return KDA_ERR_UNSUPPORTED_SHAPE;
    if (!valid_dtype(o_dtype) || !valid_dtype(b_dtype)) return KDA_ERR_UNSUPPORTED_DTYPE;
    if (f_dtype != KDA_BF16) return KDA_ERR_UNSUPPORTED_DTYPE;
    if (alog_mode != KDA_ALOG_PER_HEAD && alog_mode != KDA_ALOG_PER_CHANNEL &&
        alog_mode != KDA_ALOG_PER_HEAD_CHANNEL)
        return KDA_ERR_INVALID_ARG;
    if (cu_seqlens == nullptr && B != 1) return KDA_ERR_INVALID_ARG;
    if (A_log == nullptr || dt_bias == nullptr) return KDA_ERR_INVALID_ARG;
    if (N > 0 && (q == nullptr || k == nullptr || v == nullptr || f == nullptr || b == nullptr ||
                  o == nullptr))
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(f) || !aligned16(b) ||
        !aligned16(A_log) || !aligned16(dt_bias) || !aligned16(o) || !aligned16(initial_state) ||
        !aligned16(final_state) || !aligned16(workspace) || !aligned16(cu_seqlens))
        return KDA_ERR_MISALIGNED;
    const size_t need = kda::prefill_workspace_bytes(N, B, H);
    if (workspace_bytes < need || (need > 0 && workspace == nullptr))
        return KDA_ERR_WORKSPACE_TOO_SMALL;
    DeviceInfo *dev = nullptr;
    kda_status st = current_device(&dev);
    if (st != KDA_OK) return st;
    return from_cuda(kda::launch_prefill_gated(
        static_cast<const __nv_bfloat16 *>(q), static_cast<const __nv_bfloat16 *>(k),
        static_cast<const __nv_bfloat16 *>(v), static_cast<const __nv_bfloat16 *>(f), b,
        b_dtype == KDA_BF16, A_log, static_cast<int>(alog_mode), dt_bias, cu_seqlens, B, N, H,
        scale, initial_state, final_state, o, o_dtype == KDA_BF16, workspace, dev->error_word,
        dev->num_sms, static_cast<cudaStream_t>(stream)));
}

kda_status kda_chunk_prefill_noalloc(const void *q, const void *k, const void *v, const float *g,
                                     const float *beta, const int32_t *cu_seqlens, int B,
                                     int64_t N, int H, int K, int V, float scale,
                                     const float *initial_state, float *final_state, void *o,
                                     kda_dtype o_dtype, void *stream) {
    // The same argument and device checks as kda_chunk_prefill, in the same
    // order, before the scratch lookup, so both return the same status codes.
    kda_status st = check_prefill_args(q, k, v, g, beta, cu_seqlens, B, N, H, K, V, initial_state,
                                       final_state, o, o_dtype);
    if (st != KDA_OK) return st;
    DeviceInfo *dev = nullptr;
    st = current_device(&dev);
    if (st != KDA_OK) return st;
    void *scratch = nullptr;
    size_t scratch_bytes = 0;
    if (kda::builtin_prefill_scratch(&scratch, &scratch_bytes) != cudaSuccess) {
        cudaGetLastError();
        return KDA_ERR_CUDA;
    }
    if (kda::prefill_workspace_bytes(N, B, H) > scratch_bytes) return KDA_ERR_WORKSPACE_TOO_SMALL;
    return kda_chunk_prefill(q, k, v, g, beta, cu_seqlens, B, N, H, K, V, scale, initial_state,
                             final_state, o, o_dtype, scratch, scratch_bytes, stream);
}

kda_status kda_recurrent_decode(const void *q, const void *k, const void *v, const float *g,
                                const float *beta, float *state, int B, int H, int K, int V,
                                float scale, void *o, kda_dtype o_dtype, void *stream) {
    if (B < 0 || H < 1) return KDA_ERR_INVALID_ARG;
    if (K != 128 || V != 128) return KDA_ERR_UNSUPPORTED_SHAPE;
    if (!valid_dtype(o_dtype)) return KDA_ERR_UNSUPPORTED_DTYPE;
    if (B > 0 && (q == nullptr || k == nullptr || v == nullptr || g == nullptr ||
                  beta == nullptr || state == nullptr || o == nullptr))
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(beta) ||
        !aligned16(state) || !aligned16(o))
        return KDA_ERR_MISALIGNED;
    if (B == 0) return KDA_OK;
    DeviceInfo *dev = nullptr;
    kda_status st = current_device(&dev);
    if (st != KDA_OK) return st;
    return from_cuda(kda::launch_decode(
        static_cast<const __nv_bfloat16 *>(q), static_cast<const __nv_bfloat16 *>(k),
        static_cast<const __nv_bfloat16 *>(v), g, beta, state, B, H, scale, o,
        o_dtype == KDA_BF16, static_cast<cudaStream_t>(stream)));
}

kda_status kda_recurrent_decode_indexed(const void *q, const void *k, const void *v,
                                        const float *g, const float *beta, void *state_pool,
                                        kda_dtype state_dtype, const int32_t *state_indices,
                                        int num_slots, int B, int H, int K, int V, float scale,
                                        void *o, kda_dtype o_dtype, void *stream) {
    if (B < 0 || H < 1 || num_slots < 0) return KDA_ERR_INVALID_ARG;
    if (K != 128 || V != 128) return KDA_ERR_UNSUPPORTED_SHAPE;
    if (!valid_dtype(o_dtype) || !valid_dtype(state_dtype)) return KDA_ERR_UNSUPPORTED_DTYPE;
    if (B > 0 && (q == nullptr || k == nullptr || v == nullptr || g == nullptr ||
                  beta == nullptr || state_pool == nullptr || state_indices == nullptr ||
                  o == nullptr))
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(beta) ||
        !aligned16(state_pool) || !aligned16(state_indices) || !aligned16(o))
        return KDA_ERR_MISALIGNED;
    if (B == 0) return KDA_OK;
    DeviceInfo *dev = nullptr;
    kda_status st = current_device(&dev);
    if (st != KDA_OK) return st;
    return from_cuda(kda::launch_decode_indexed(
        static_cast<const __nv_bfloat16 *>(q), static_cast<const __nv_bfloat16 *>(k),
        static_cast<const __nv_bfloat16 *>(v), g, beta, state_pool, state_dtype == KDA_BF16,
        state_indices, num_slots, B, H, scale, o, o_dtype == KDA_BF16, dev->error_word,
        static_cast<cudaStream_t>(stream)));
}

kda_status kda_recurrent_decode_gated(const void *q, const void *k, const void *v,
                                      const void *f, kda_dtype f_dtype, const void *b,
                                      kda_dtype b_dtype, const float *A_log,
                                      kda_alog_mode alog_mode, const float *dt_bias,
                                      void *state_pool, kda_dtype state_dtype,
                                      const int32_t *state_indices, int num_slots, int B, int H,
                                      int K, int V, float scale, void *o, kda_dtype o_dtype,
                                      void *stream) {
    if (B < 0 || H < 1 || num_slots < 0) return KDA_ERR_INVALID_ARG;
    if (state_indices == nullptr && num_slots < B) return KDA_ERR_INVALID_ARG;
    if (K != 128 || V != 128) return KDA_ERR_UNSUPPORTED_SHAPE;
    if (!valid_dtype(o_dtype) || !valid_dtype(state_dtype) || !valid_dtype(f_dtype) ||
        !valid_dtype(b_dtype))
        return KDA_ERR_UNSUPPORTED_DTYPE;
    if (alog_mode != KDA_ALOG_PER_HEAD && alog_mode != KDA_ALOG_PER_CHANNEL &&
        alog_mode != KDA_ALOG_PER_HEAD_CHANNEL)
        return KDA_ERR_INVALID_ARG;
    if (B > 0 && (q == nullptr || k == nullptr || v == nullptr || f == nullptr || b == nullptr ||
                  A_log == nullptr || dt_bias == nullptr || state_pool == nullptr ||
                  o == nullptr))
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(f) || !aligned16(b) ||
        !aligned16(state_pool) || !aligned16(state_indices) || !aligned16(o))
        return KDA_ERR_MISALIGNED;
    if (B == 0) return KDA_OK;
    DeviceInfo *dev = nullptr;
    kda_status st = current_device(&dev);
    if (st != KDA_OK) return st;
    return from_cuda(kda::launch_decode_gated(
        static_cast<const __nv_bfloat16 *>(q), static_cast<const __nv_bfloat16 *>(k),
        static_cast<const __nv_bfloat16 *>(v), f, f_dtype == KDA_BF16, b, b_dtype == KDA_BF16,
        A_log, static_cast<int>(alog_mode), dt_bias, state_pool, state_dtype == KDA_BF16,
        state_indices, state_indices == nullptr ? B : num_slots, B, H, scale, o,
        o_dtype == KDA_BF16, dev->error_word, static_cast<cudaStream_t>(stream)));
}

size_t kda_gate_backward_workspace_size(int64_t N, int H, int K) {
    return kda::gate_bwd_workspace_bytes(N, H, K);
}

kda_status kda_gate_backward(const void *f, kda_dtype f_dtype, const void *b, kda_dtype b_dtype,
                             const float *A_log, kda_alog_mode alog_mode, const float *dt_bias,
                             const float *dg, const float *dbeta, float *df, float *db,
                             float *dA_log, float *ddt_bias, int64_t N, int H, int K,
                             void *workspace, size_t workspace_bytes, void *stream) {
    if (N < 0 || H < 1 || K < 1) return KDA_ERR_INVALID_ARG;
    if (K % 8 != 0) return KDA_ERR_UNSUPPORTED_SHAPE;
    if (!valid_dtype(f_dtype) || !valid_dtype(b_dtype)) return KDA_ERR_UNSUPPORTED_DTYPE;
    if (alog_mode != KDA_ALOG_PER_HEAD && alog_mode != KDA_ALOG_PER_CHANNEL &&
        alog_mode != KDA_ALOG_PER_HEAD_CHANNEL)
        return KDA_ERR_INVALID_ARG;
    const bool with_beta = b != nullptr;
    if (with_beta != (dbeta != nullptr) || with_beta != (db != nullptr)) return KDA_ERR_INVALID_ARG;
    if (A_log == nullptr || dt_bias == nullptr) return KDA_ERR_INVALID_ARG;
    if (N > 0 && (f == nullptr || dg == nullptr || df == nullptr)) return KDA_ERR_INVALID_ARG;
    if (!aligned16(f) || !aligned16(dg) || !aligned16(df) || !aligned16(workspace))
        return KDA_ERR_MISALIGNED;
    if (workspace == nullptr || workspace_bytes < kda::gate_bwd_workspace_bytes(N, H, K))
        return KDA_ERR_WORKSPACE_TOO_SMALL;
    DeviceInfo *dev = nullptr;
    kda_status st = current_device(&dev);
    if (st != KDA_OK) return st;
    return from_cuda(kda::launch_gate_backward(
        f, f_dtype == KDA_BF16, b, b_dtype == KDA_BF16, A_log, static_cast<int>(alog_mode),
        dt_bias, dg, dbeta, df, db, dA_log, ddt_bias, N, H, K, workspace,
        static_cast<cudaStream_t>(stream)));
}

kda_status kda_short_conv_qkv(const void *x_q, const void *x_k, const void *x_v,
                              const float *w_q, const float *w_k, const float *w_v,
                              const int32_t *cu_seqlens, int B, int64_t N, int C,
                              const void *conv_state_in, void *conv_state_out,
                              void *q, void *k, void *v, void *stream) {
    if (N < 0 || B < 1 || (cu_seqlens == nullptr && B != 1)) return KDA_ERR_INVALID_ARG;
    if (C < 128 || C % 128 != 0) return KDA_ERR_UNSUPPORTED_SHAPE;
    const void *xs[3] = {x_q, x_k, x_v};
    const float *ws[3] = {w_q, w_k, w_v};
    void *ys[3] = {q, k, v};
    const size_t tok_bytes = static_cast<size_t>(N) * C * 2;
    const size_t st_bytes = static_cast<size_t>(B) * 9 * C * 2;
    if (N > 0) {
        for (int i = 0; i < 3; ++i)
            if (xs[i] == nullptr || ws[i] == nullptr || ys[i] == nullptr) return KDA_ERR_INVALID_ARG;
        for (int i = 0; i < 3; ++i)
            for (int j = 0; j < 3; ++j) {
                if (overlaps(ys[i], tok_bytes, xs[j], tok_bytes)) return KDA_ERR_INVALID_ARG;
                if (i < j && overlaps(ys[i], tok_bytes, ys[j], tok_bytes)) return KDA_ERR_INVALID_ARG;
            }
    }
    if (overlaps(conv_state_in, st_bytes, conv_state_out, st_bytes)) return KDA_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i)
        if (!aligned16(xs[i]) || !aligned16(ws[i]) || !aligned16(ys[i])) return KDA_ERR_MISALIGNED;
    if (!aligned16(conv_state_in) || !aligned16(conv_state_out) || !aligned16(cu_seqlens))
        return KDA_ERR_MISALIGNED;
    if (N == 0 && conv_state_out == nullptr) return KDA_OK;
    DeviceInfo *dev = nullptr;
    kda_status st = current_device(&dev);
    if (st != KDA_OK) return st;
    const __nv_bfloat16 *xb[3];
    __nv_bfloat16 *yb[3];
    for (int i = 0; i < 3; ++i) {
        xb[i] = static_cast<const __nv_bfloat16 *>(xs[i]);
        yb[i] = static_cast<__nv_bfloat16 *>(ys[i]);
    }
    return from_cuda(kda::launch_short_conv(
        xb, ws, yb, cu_seqlens, B, N, C, static_cast<const __nv_bfloat16 *>(conv_state_in),
        static_cast<__nv_bfloat16 *>(conv_state_out), dev->error_word,
        static_cast<cudaStream_t>(stream)));
}

kda_status kda_short_conv_qkv_step(const void *x_q, const void *x_k, const void *x_v,
                                   const float *w_q, const float *w_k, const float *w_v,
                                   void *conv_state_pool, const int32_t *state_indices,
                                   int num_slots, int B, int C,
                                   void *q, void *k, void *v, void *stream) {
    if (B < 0 || B > 65535 || num_slots < 0) return KDA_ERR_INVALID_ARG;
    if (state_indices == nullptr && num_slots < B) return KDA_ERR_INVALID_ARG;
    if (C < 128 || C % 128 != 0) return KDA_ERR_UNSUPPORTED_SHAPE;
    const void *xs[3] = {x_q, x_k, x_v};
    const float *ws[3] = {w_q, w_k, w_v};
    void *ys[3] = {q, k, v};
    if (B > 0) {
        for (int i = 0; i < 3; ++i)
            if (xs[i] == nullptr || ws[i] == nullptr || ys[i] == nullptr) return KDA_ERR_INVALID_ARG;
        if (conv_state_pool == nullptr) return KDA_ERR_INVALID_ARG;
    }
    for (int i = 0; i < 3; ++i)
        if (!aligned16(xs[i]) || !aligned16(ws[i]) || !aligned16(ys[i])) return KDA_ERR_MISALIGNED;
    if (!aligned16(conv_state_pool) || !aligned16(state_indices)) return KDA_ERR_MISALIGNED;
    if (B == 0) return KDA_OK;
    DeviceInfo *dev = nullptr;
    kda_status st = current_device(&dev);
    if (st != KDA_OK) return st;
    const __nv_bfloat16 *xb[3];
    __nv_bfloat16 *yb[3];
    for (int i = 0; i < 3; ++i) {
        xb[i] = static_cast<const __nv_bfloat16 *>(xs[i]);
        yb[i] = static_cast<__nv_bfloat16 *>(ys[i]);
    }
    return from_cuda(kda::launch_short_conv_step(
        xb, ws, yb, static_cast<__nv_bfloat16 *>(conv_state_pool), state_indices, num_slots, B, C,
        dev->error_word, static_cast<cudaStream_t>(stream)));
}

size_t kda_recurrent_backward_workspace_size(int64_t N, int B, int H, int K, int V) {
    if (N < 0 || B < 1 || H < 1 || K != 128 || V != 128) return 0;
    return kda::backward_workspace_bytes(N, B, H, kda::backward_ctas(B, H, kda::kBackwardMaxCtas));
}

kda_status kda_recurrent_backward(const void *q, const void *k, const void *v, const float *g,
                                  const float *beta, const int32_t *cu_seqlens, int B, int64_t N,
                                  int H, int K, int V, float scale, const float *initial_state,
                                  const void *dO, kda_dtype dO_dtype, const float *dS_final,
                                  float *dq, float *dk, float *dv, float *dg, float *dbeta,
                                  float *dS0, void *workspace, size_t workspace_bytes,
                                  void *stream) {
    if (N < 0 || B < 1 || H < 1) return KDA_ERR_INVALID_ARG;
    if (K != 128 || V != 128) return KDA_ERR_UNSUPPORTED_SHAPE;
    if (!valid_dtype(dO_dtype)) return KDA_ERR_UNSUPPORTED_DTYPE;
    if (cu_seqlens == nullptr && B != 1) return KDA_ERR_INVALID_ARG;
    if (N > 0 && (q == nullptr || k == nullptr || v == nullptr || g == nullptr ||
                  beta == nullptr || dO == nullptr || dq == nullptr || dk == nullptr ||
                  dv == nullptr || dg == nullptr || dbeta == nullptr))
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(beta) ||
        !aligned16(dO) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned16(dg) ||
        !aligned16(dbeta) || !aligned16(initial_state) || !aligned16(dS_final) ||
        !aligned16(dS0) || !aligned16(workspace) || !aligned16(cu_seqlens))
        return KDA_ERR_MISALIGNED;
    const size_t need = kda_recurrent_backward_workspace_size(N, B, H, K, V);
    if (workspace_bytes < need || workspace == nullptr) return KDA_ERR_WORKSPACE_TOO_SMALL;
    DeviceInfo *dev = nullptr;
    kda_status st = current_device(&dev);
    if (st != KDA_OK) return st;
    const int ctas = kda::backward_ctas(B, H, dev->num_sms < kda::kBackwardMaxCtas
                                                  ? dev->num_sms : kda::kBackwardMaxCtas);
    return from_cuda(kda::launch_backward(
        static_cast<const __nv_bfloat16 *>(q), static_cast<const __nv_bfloat16 *>(k),
        static_cast<const __nv_bfloat16 *>(v), g, beta, cu_seqlens, B, N, H, scale, initial_state,
        dO, dO_dtype == KDA_BF16, dS_final, dq, dk, dv, dg, dbeta, dS0, workspace, ctas,
        dev->error_word, static_cast<cudaStream_t>(stream)));
}

size_t kda_chunk_backward_workspace_size(int64_t N, int B, int H, int K, int V) {
    if (N < 0 || B < 1 || H < 1 || K != 128 || V != 128) return 0;
    const int64_t chains = static_cast<int64_t>(B) * H;
    const int ctas = static_cast<int>(chains < kda::kChunkBwdMaxCtas ? chains : kda::kChunkBwdMaxCtas);
    return kda::chunk_bwd_workspace_bytes(N, B, H, ctas);
}

kda_status kda_chunk_backward(const void *q, const void *k, const void *v, const float *g,
                              const float *beta, const int32_t *cu_seqlens, int B, int64_t N,
                              int H, int K, int V, float scale, const float *initial_state,
                              const void *dO, kda_dtype dO_dtype, const float *dS_final,
                              float *dq, float *dk, float *dv, float *dg, float *dbeta,
                              float *dS0, void *workspace, size_t workspace_bytes, void *stream) {
    if (N < 0 || B < 1 || H < 1) return KDA_ERR_INVALID_ARG;
    if (K != 128 || V != 128) return KDA_ERR_UNSUPPORTED_SHAPE;
    if (!valid_dtype(dO_dtype)) return KDA_ERR_UNSUPPORTED_DTYPE;
    if (cu_seqlens == nullptr && B != 1) return KDA_ERR_INVALID_ARG;
    if (N > 0 && (q == nullptr || k == nullptr || v == nullptr || g == nullptr ||
                  beta == nullptr || dO == nullptr || dq == nullptr || dk == nullptr ||
                  dv == nullptr || dg == nullptr || dbeta == nullptr))
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(beta) ||
        !aligned16(dO) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned16(dg) ||
        !aligned16(dbeta) || !aligned16(initial_state) || !aligned16(dS_final) ||
        !aligned16(dS0) || !aligned16(workspace) || !aligned16(cu_seqlens))
        return KDA_ERR_MISALIGNED;
    const size_t need = kda_chunk_backward_workspace_size(N, B, H, K, V);
    if (workspace_bytes < need || workspace == nullptr) return KDA_ERR_WORKSPACE_TOO_SMALL;
    DeviceInfo *dev = nullptr;
    kda_status st = current_device(&dev);
    if (st != KDA_OK) return st;
    const int64_t chains = static_cast<int64_t>(B) * H;
    int ctas = dev->num_sms < kda::kChunkBwdMaxCtas ? dev->num_sms : kda::kChunkBwdMaxCtas;
    if (chains < ctas) ctas = static_cast<int>(chains);
    return from_cuda(kda::launch_chunk_backward(
        static_cast<const __nv_bfloat16 *>(q), static_cast<const __nv_bfloat16 *>(k),
        static_cast<const __nv_bfloat16 *>(v), g, beta, cu_seqlens, B, N, H, scale, initial_state,
        dO, dO_dtype == KDA_BF16, dS_final, dq, dk, dv, dg, dbeta, dS0, workspace, ctas,
        dev->error_word, dev->num_sms, static_cast<cudaStream_t>(stream)));
}

size_t kda_chunk_checkpoints_size(int64_t N, int B, int H, int K, int V) {
    if (N < 0 || B < 1 || H < 1 || K != 128 || V != 128) return 0;
    return kda::chunk_checkpoints_bytes(N, B, H);
}

kda_status kda_chunk_prefill_checkpointed(const void *q, const void *k, const void *v,
                                          const float *g, const float *beta,
                                          const int32_t *cu_seqlens, int B, int64_t N, int H,
                                          int K, int V, float scale, const float *initial_state,
                                          float *final_state, void *o, kda_dtype o_dtype,
                                          void *checkpoints, size_t checkpoints_bytes,
                                          void *workspace, size_t workspace_bytes, void *stream) {
    kda_status st = check_prefill_args(q, k, v, g, beta, cu_seqlens, B, N, H, K, V, initial_state,
                                       final_state, o, o_dtype);
    if (st != KDA_OK) return st;
    if (!aligned16(workspace) || !aligned16(checkpoints)) return KDA_ERR_MISALIGNED;
    const size_t need = kda::prefill_workspace_bytes(N, B, H);
    if (workspace_bytes < need || (need > 0 && workspace == nullptr))
        return KDA_ERR_WORKSPACE_TOO_SMALL;
    if (checkpoints == nullptr || checkpoints_bytes < kda::chunk_checkpoints_bytes(N, B, H))
        return KDA_ERR_WORKSPACE_TOO_SMALL;
    DeviceInfo *dev = nullptr;
    st = current_device(&dev);
    if (st != KDA_OK) return st;
    uint8_t *cp = static_cast<uint8_t *>(checkpoints);
    return from_cuda(kda::launch_prefill_checkpointed(
        static_cast<const __nv_bfloat16 *>(q), static_cast<const __nv_bfloat16 *>(k),
        static_cast<const __nv_bfloat16 *>(v), g, beta, cu_seqlens, B, N, H, scale, initial_state,
        final_state, o, o_dtype == KDA_BF16,
        reinterpret_cast<float *>(cp + kda::chunk_checkpoint_flags_bytes(B, H)),
        reinterpret_cast<int *>(cp), workspace, dev->error_word, dev->num_sms,
        static_cast<cudaStream_t>(stream)));
}

size_t kda_chunk_backward_checkpointed_workspace_size(int64_t N, int B, int H, int K, int V) {
    if (N < 0 || B < 1 || H < 1 || K != 128 || V != 128) return 0;
    const int64_t chains = static_cast<int64_t>(B) * H;
    const int ctas = static_cast<int>(chains < kda::kChunkBwdMaxCtas ? chains : kda::kChunkBwdMaxCtas);
    return kda::chunk_bwd_from_checkpoints_workspace_bytes(ctas);
}

kda_status kda_chunk_backward_checkpointed(const void *q, const void *k, const void *v,
                                           const float *g, const float *beta,
                                           const int32_t *cu_seqlens, int B, int64_t N, int H,
                                           int K, int V, float scale, const void *checkpoints,
                                           size_t checkpoints_bytes, const void *dO,
                                           kda_dtype dO_dtype, const float *dS_final, float *dq,
                                           float *dk, float *dv, float *dg, float *dbeta,
                                           float *dS0, void *workspace, size_t workspace_bytes,
                                           void *stream) {
    if (N < 0 || B < 1 || H < 1) return KDA_ERR_INVALID_ARG;
    if (K != 128 || V != 128) return KDA_ERR_UNSUPPORTED_SHAPE;
    if (!valid_dtype(dO_dtype)) return KDA_ERR_UNSUPPORTED_DTYPE;
    if (cu_seqlens == nullptr && B != 1) return KDA_ERR_INVALID_ARG;
    if (N > 0 && (q == nullptr || k == nullptr || v == nullptr || g == nullptr ||
                  beta == nullptr || dO == nullptr || dq == nullptr || dk == nullptr ||
                  dv == nullptr || dg == nullptr || dbeta == nullptr))
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(beta) ||
        !aligned16(dO) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned16(dg) ||
        !aligned16(dbeta) || !aligned16(checkpoints) || !aligned16(dS_final) ||
        !aligned16(dS0) || !aligned16(workspace) || !aligned16(cu_seqlens))
        return KDA_ERR_MISALIGNED;
    if (checkpoints == nullptr || checkpoints_bytes < kda::chunk_checkpoints_bytes(N, B, H))
        return KDA_ERR_WORKSPACE_TOO_SMALL;
    const size_t need = kda_chunk_backward_checkpointed_workspace_size(N, B, H, K, V);
    if (workspace_bytes < need || workspace == nullptr) return KDA_ERR_WORKSPACE_TOO_SMALL;
    DeviceInfo *dev = nullptr;
    kda_status st = current_device(&dev);
    if (st != KDA_OK) return st;
    const int64_t chains = static_cast<int64_t>(B) * H;
    int ctas = dev->num_sms < kda::kChunkBwdMaxCtas ? dev->num_sms : kda::kChunkBwdMaxCtas;
    if (chains < ctas) ctas = static_cast<int>(chains);
    return from_cuda(kda::launch_chunk_backward_from_checkpoints(
        static_cast<const __nv_bfloat16 *>(q), static_cast<const __nv_bfloat16 *>(k),
        static_cast<const __nv_bfloat16 *>(v), g, beta, cu_seqlens, B, N, H, scale, checkpoints,
        dO, dO_dtype == KDA_BF16, dS_final, dq, dk, dv, dg, dbeta, dS0, workspace, ctas,
        dev->error_word, static_cast<cudaStream_t>(stream)));
}

kda_status kda_page_plan(const int32_t *cached_lens, const int32_t *new_lens,
                         const int32_t *free_pages, int num_free, int32_t *block_table,
                         int max_pages, int B, int page_size, int num_pages, int32_t *seq_lens,
                         int32_t *cu_seqlens, int32_t *slot_map, int64_t N, int32_t *pages_used,
                         void *stream) {
    if (B < 0 || N < 0 || N > INT32_MAX || num_free < 0 || max_pages < 0 || page_size < 1 ||
        num_pages < 0)
        return KDA_ERR_INVALID_ARG;
    if (static_cast<int64_t>(num_pages) * page_size > INT32_MAX) return KDA_ERR_UNSUPPORTED_SHAPE;
    if (cu_seqlens == nullptr || pages_used == nullptr || (N > 0 && slot_map == nullptr) ||
        (num_free > 0 && free_pages == nullptr))
        return KDA_ERR_INVALID_ARG;
    if (B > 0 && (cached_lens == nullptr || new_lens == nullptr || seq_lens == nullptr ||
                  (max_pages > 0 && block_table == nullptr)))
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(cached_lens) || !aligned16(new_lens) ||
        (reinterpret_cast<uintptr_t>(free_pages) & 3u) != 0 || !aligned16(block_table) || !aligned16(seq_lens) || !aligned16(cu_seqlens) ||
        !aligned16(slot_map) || !aligned16(pages_used))
        return KDA_ERR_MISALIGNED;
    // every CTA reads the lists while others write the results
    const size_t rows = static_cast<size_t>(B) * 4;
    const struct {
        const void *p;
        size_t bytes;
    } bufs[] = {{seq_lens, rows},
                {cu_seqlens, rows + 4},
                {slot_map, static_cast<size_t>(N) * 4},
                {pages_used, 4},
                {block_table, rows * static_cast<size_t>(max_pages)},
                {cached_lens, rows},
                {new_lens, rows},
                {free_pages, static_cast<size_t>(num_free) * 4}};
    for (int i = 0; i < 5; ++i)
        for (int j = i + 1; j < 8; ++j)
            if (overlaps(bufs[i].p, bufs[i].bytes, bufs[j].p, bufs[j].bytes))
                return KDA_ERR_INVALID_ARG;
    DeviceInfo *dev = nullptr;
    kda_status st = current_device(&dev);
    if (st != KDA_OK) return st;
    return from_cuda(kda::launch_page_plan(cached_lens, new_lens, free_pages, num_free, block_table,
                                           max_pages, B, page_size, num_pages, seq_lens, cu_seqlens,
                                           slot_map, N, pages_used, dev->error_word,
                                           static_cast<cudaStream_t>(stream)));
}

kda_status kda_paged_append(const void *k, const void *v, int64_t k_row_stride,
                            int64_t v_row_stride, const int32_t *slot_map, int64_t N,
                            const kda_paged_cache *cache, void *stream) {
    kda::PagedView view;
    kda_status st = paged_view(cache, &view);
    if (st != KDA_OK) return st;
    if (N < 0 || N > INT32_MAX || view.k == view.v) return KDA_ERR_INVALID_ARG;
    if (N > 0 && (k == nullptr || v == nullptr || slot_map == nullptr)) return KDA_ERR_INVALID_ARG;
    const int64_t width = static_cast<int64_t>(view.heads) * view.head_dim;
    if (N > 1 && (k_row_stride < width || v_row_stride < width)) return KDA_ERR_INVALID_ARG;
    if (k_row_stride > INT64_MAX / 4 / (N + 1) || v_row_stride > INT64_MAX / 4 / (N + 1))
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(slot_map) ||
        (N > 1 && (k_row_stride % 8 != 0 || v_row_stride % 8 != 0)))
        return KDA_ERR_MISALIGNED;
    if (N == 0) return KDA_OK;
    DeviceInfo *dev = nullptr;
    st = current_device(&dev);
    if (st != KDA_OK) return st;
    return from_cuda(kda::launch_paged_append(
        static_cast<const __nv_bfloat16 *>(k), static_cast<const __nv_bfloat16 *>(v), k_row_stride,
        v_row_stride, slot_map, N, view, dev->error_word, static_cast<cudaStream_t>(stream)));
}

size_t kda_paged_decode_workspace_size(int B, int q_heads, int kv_heads, int head_dim) {
    if (B < 0 || kv_heads < 1 || q_heads < 1 ||
        (head_dim != 64 && head_dim != 128 && head_dim != 256) ||
        !paged_decode_sizes(B, q_heads, kv_heads, head_dim))
        return 0;
    return kda::paged_decode_workspace_bytes(B, q_heads, kv_heads, head_dim);
}

kda_status kda_paged_decode(const void *q, int64_t q_row_stride, const kda_paged_cache *cache,
                            const int32_t *block_table, int max_pages, const int32_t *seq_lens,
                            int B, int q_heads, float scale, void *o, kda_dtype o_dtype,
                            float *lse, void *workspace, size_t workspace_bytes, void *stream) {
    kda::PagedView view;
    kda_status st = paged_view(cache, &view);
    if (st != KDA_OK) return st;
    if (B < 0 || max_pages < 0 || q_heads < 1) return KDA_ERR_INVALID_ARG;
    if (!paged_decode_sizes(B, q_heads, view.heads, view.head_dim)) return KDA_ERR_UNSUPPORTED_SHAPE;
    const int64_t width = static_cast<int64_t>(q_heads) * view.head_dim;
    if (!valid_dtype(o_dtype)) return KDA_ERR_UNSUPPORTED_DTYPE;
    if (B > 0 && (q == nullptr || seq_lens == nullptr || o == nullptr ||
                  (max_pages > 0 && block_table == nullptr)))
        return KDA_ERR_INVALID_ARG;
    if (B > 1 && (q_row_stride < width || q_row_stride > INT64_MAX / 4 / B))
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(block_table) || !aligned16(seq_lens) || !aligned16(o) ||
        !aligned16(lse) || !aligned16(workspace) || (B > 1 && q_row_stride % 8 != 0))
        return KDA_ERR_MISALIGNED;
    const size_t need = kda::paged_decode_workspace_bytes(B, q_heads, view.heads, view.head_dim);
    if (workspace_bytes < need || (need > 0 && workspace == nullptr))
        return KDA_ERR_WORKSPACE_TOO_SMALL;
    if (B == 0) return KDA_OK;
    DeviceInfo *dev = nullptr;
    st = current_device(&dev);
    if (st != KDA_OK) return st;
    try {
        return from_cuda(kda::launch_paged_decode(
            static_cast<const __nv_bfloat16 *>(q), q_row_stride, view, block_table, max_pages,
            seq_lens, B, q_heads, scale, o, o_dtype == KDA_BF16, lse, workspace, dev->error_word,
            dev->num_sms, static_cast<cudaStream_t>(stream)));
    } catch (...) {  // the list of kernels with raised shared-memory limits could not grow
        return KDA_ERR_CUDA;
    }
}

kda_status kda_recurrent_tree_decode(const void *q, const void *k, const void *v, const float *g,
                                     const float *beta, const void *state_pool,
                                     kda_dtype state_dtype, const int32_t *state_indices,
                                     int num_slots, const int32_t *cu_seqlens,
                                     const uint64_t *ancestors, int B, int64_t N, int max_nodes,
                                     int H, int K, int V, float scale, void *o, kda_dtype o_dtype,
                                     float *u, void *stream) {
    kda_status st = tree_sizes(B, N, max_nodes, num_slots, state_indices);
    if (st != KDA_OK) return st;
    if (H < 1) return KDA_ERR_INVALID_ARG;
    if (K != 128 || V != 128 || static_cast<int64_t>(B) * H > INT32_MAX)
        return KDA_ERR_UNSUPPORTED_SHAPE;
    if (!valid_dtype(o_dtype) || !valid_dtype(state_dtype)) return KDA_ERR_UNSUPPORTED_DTYPE;
    if (B == 0) return KDA_OK;
    if (cu_seqlens == nullptr || state_pool == nullptr ||
        (N > 0 && (q == nullptr || k == nullptr || v == nullptr || g == nullptr ||
                   beta == nullptr || ancestors == nullptr || o == nullptr)))
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(beta) ||
        !aligned16(state_pool) || !aligned16(state_indices) || !aligned16(cu_seqlens) ||
        !aligned16(ancestors) || !aligned16(o) || !aligned16(u))
        return KDA_ERR_MISALIGNED;
    const size_t values = static_cast<size_t>(N) * H * 128;
    const size_t o_bytes = values * (o_dtype == KDA_BF16 ? 2 : 4);
    const size_t pool = static_cast<size_t>(num_slots) * H * 16384 * (state_dtype == KDA_BF16 ? 2 : 4);
    const Buffer ins[] = {{q, values * 2}, {k, values * 2}, {v, values * 2}, {g, values * 4}, {state_pool, pool},
                          {beta, static_cast<size_t>(N) * H * 4}, {state_indices, static_cast<size_t>(B) * 4},
                          {cu_seqlens, static_cast<size_t>(B) * 4 + 4}, {ancestors, static_cast<size_t>(N) * 8}};
    for (const Buffer &in : ins)
        if (overlaps(o, o_bytes, in.p, in.bytes) || overlaps(u, values * 4, in.p, in.bytes))
            return KDA_ERR_INVALID_ARG;
    if (overlaps(o, o_bytes, u, values * 4)) return KDA_ERR_INVALID_ARG;
    DeviceInfo *dev = nullptr;
    st = current_device(&dev);
    if (st != KDA_OK) return st;
    kda::TreeStep a = {};
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k = static_cast<const __nv_bfloat16 *>(k);
    a.v = static_cast<const __nv_bfloat16 *>(v);
    a.g = g;
    a.beta = beta;
    a.pool = const_cast<void *>(state_pool);
    a.slots = state_indices;
    a.num_slots = num_slots;
    a.cu = cu_seqlens;
    a.ancestors = ancestors;
    a.B = B;
    a.H = H;
    a.max_nodes = max_nodes;
    a.N = N;
    a.scale = scale;
    a.o = o;
    a.u = u;
    a.err = dev->error_word;
    try {
        return from_cuda(kda::launch_tree_decode(a, state_dtype == KDA_BF16, o_dtype == KDA_BF16, dev->num_sms,
                                                 static_cast<cudaStream_t>(stream)));
    } catch (...) {  // the list of kernels with raised shared-memory limits could not grow
        return KDA_ERR_CUDA;
    }
}

kda_status kda_recurrent_tree_commit(const void *k, const float *g, const float *u,
                                     void *state_pool, kda_dtype state_dtype,
                                     const int32_t *state_indices, int num_slots,
                                     const int32_t *cu_seqlens, const uint64_t *ancestors,
                                     const int32_t *last, int B, int64_t N, int max_nodes, int H,
                                     int K, int V, void *stream) {
    kda_status st = tree_sizes(B, N, max_nodes, num_slots, state_indices);
    if (st != KDA_OK) return st;
    if (H < 1) return KDA_ERR_INVALID_ARG;
    if (K != 128 || V != 128 || static_cast<int64_t>(B) * H > INT32_MAX)
        return KDA_ERR_UNSUPPORTED_SHAPE;
    if (!valid_dtype(state_dtype)) return KDA_ERR_UNSUPPORTED_DTYPE;
    if (B == 0) return KDA_OK;
    if (cu_seqlens == nullptr || state_pool == nullptr || last == nullptr ||
        (N > 0 && (k == nullptr || g == nullptr || u == nullptr || ancestors == nullptr)))
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(g) || !aligned16(u) || !aligned16(state_pool) ||
        !aligned16(state_indices) || !aligned16(cu_seqlens) || !aligned16(ancestors) ||
        !aligned16(last))
        return KDA_ERR_MISALIGNED;
    DeviceInfo *dev = nullptr;
    st = current_device(&dev);
    if (st != KDA_OK) return st;
    kda::TreeStep a = {};
    a.k = static_cast<const __nv_bfloat16 *>(k);
    a.g = g;
    a.pool = state_pool;
    a.slots = state_indices;
    a.num_slots = num_slots;
    a.cu = cu_seqlens;
    a.ancestors = ancestors;
    a.last = last;
    a.B = B;
    a.H = H;
    a.max_nodes = max_nodes;
    a.N = N;
    a.u = const_cast<float *>(u);
    a.err = dev->error_word;
    return from_cuda(kda::launch_tree_commit(a, state_dtype == KDA_BF16, static_cast<cudaStream_t>(stream)));
}

kda_status kda_short_conv_qkv_tree(const void *x_q, const void *x_k, const void *x_v,
                                   const float *w_q, const float *w_k, const float *w_v,
                                   const void *conv_state_pool, const int32_t *state_indices,
                                   int num_slots, const int32_t *cu_seqlens,
                                   const uint64_t *ancestors, int B, int64_t N, int max_nodes,
                                   int C, void *q, void *k, void *v, void *stream) {
    kda_status st = tree_sizes(B, N, max_nodes, num_slots, state_indices);
    if (st != KDA_OK) return st;
    if (C < 128 || C % 128 != 0) return KDA_ERR_UNSUPPORTED_SHAPE;
    if (B == 0) return KDA_OK;
    if (cu_seqlens == nullptr || conv_state_pool == nullptr || (N > 0 && ancestors == nullptr))
        return KDA_ERR_INVALID_ARG;
    const void *xs[3] = {x_q, x_k, x_v};
    const float *ws[3] = {w_q, w_k, w_v};
    void *ys[3] = {q, k, v};
    const size_t bytes = static_cast<size_t>(N) * C * 2;
    const size_t pool = static_cast<size_t>(num_slots) * 9 * C * 2;
    for (int i = 0; i < 3; ++i) {
        if (N > 0 && (xs[i] == nullptr || ws[i] == nullptr || ys[i] == nullptr))
            return KDA_ERR_INVALID_ARG;
        if (!aligned16(xs[i]) || !aligned16(ws[i]) || !aligned16(ys[i])) return KDA_ERR_MISALIGNED;
        for (int j = 0; j < 3; ++j)
            if (overlaps(ys[i], bytes, xs[j], bytes) ||
                overlaps(ys[i], bytes, ws[j], static_cast<size_t>(C) * 16) ||
                (i < j && overlaps(ys[i], bytes, ys[j], bytes)))
                return KDA_ERR_INVALID_ARG;
        const Buffer ins[] = {{conv_state_pool, pool}, {state_indices, static_cast<size_t>(B) * 4},
                              {cu_seqlens, static_cast<size_t>(B) * 4 + 4}, {ancestors, static_cast<size_t>(N) * 8}};
        for (const Buffer &in : ins)
            if (overlaps(ys[i], bytes, in.p, in.bytes)) return KDA_ERR_INVALID_ARG;
    }
    if (!aligned16(conv_state_pool) || !aligned16(state_indices) || !aligned16(cu_seqlens) ||
        !aligned16(ancestors))
        return KDA_ERR_MISALIGNED;
    DeviceInfo *dev = nullptr;
    st = current_device(&dev);
    if (st != KDA_OK) return st;
    kda::TreeConv a = {};
    for (int i = 0; i < 3; ++i) {
        a.x[i] = static_cast<const __nv_bfloat16 *>(xs[i]);
        a.w[i] = ws[i];
        a.y[i] = static_cast<__nv_bfloat16 *>(ys[i]);
    }
    a.pool = static_cast<__nv_bfloat16 *>(const_cast<void *>(conv_state_pool));
    a.slots = state_indices;
    a.num_slots = num_slots;
    a.cu = cu_seqlens;
    a.ancestors = ancestors;
    a.B = B;
    a.C = C;
    a.max_nodes = max_nodes;
    a.N = N;
    a.err = dev->error_word;
    try {
        return from_cuda(kda::launch_tree_conv(a, dev->num_sms, static_cast<cudaStream_t>(stream)));
    } catch (...) {  // the list of kernels with raised shared-memory limits could not grow
        return KDA_ERR_CUDA;
    }
}

kda_status kda_short_conv_tree_commit(const void *x_q, const void *x_k, const void *x_v,
                                      void *conv_state_pool, const int32_t *state_indices,
                                      int num_slots, const int32_t *cu_seqlens,
                                      const uint64_t *ancestors, const int32_t *last, int B,
                                      int64_t N, int max_nodes, int C, void *stream) {
    kda_status st = tree_sizes(B, N, max_nodes, num_slots, state_indices);
    if (st != KDA_OK) return st;
    if (C < 128 || C % 128 != 0) return KDA_ERR_UNSUPPORTED_SHAPE;
    if (B == 0) return KDA_OK;
    if (cu_seqlens == nullptr || conv_state_pool == nullptr || last == nullptr ||
        (N > 0 && (x_q == nullptr || x_k == nullptr || x_v == nullptr || ancestors == nullptr)))
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(x_q) || !aligned16(x_k) || !aligned16(x_v) || !aligned16(conv_state_pool) ||
        !aligned16(state_indices) || !aligned16(cu_seqlens) || !aligned16(ancestors) ||
        !aligned16(last))
        return KDA_ERR_MISALIGNED;
    DeviceInfo *dev = nullptr;
    st = current_device(&dev);
    if (st != KDA_OK) return st;
    kda::TreeConv a = {};
    a.x[0] = static_cast<const __nv_bfloat16 *>(x_q);
    a.x[1] = static_cast<const __nv_bfloat16 *>(x_k);
    a.x[2] = static_cast<const __nv_bfloat16 *>(x_v);
    a.pool = static_cast<__nv_bfloat16 *>(conv_state_pool);
    a.slots = state_indices;
    a.num_slots = num_slots;
    a.cu = cu_seqlens;
    a.ancestors = ancestors;
    a.last = last;
    a.B = B;
    a.C = C;
    a.max_nodes = max_nodes;
    a.N = N;
    a.err = dev->error_word;
    return from_cuda(kda::launch_tree_conv_commit(a, static_cast<cudaStream_t>(stream)));
}

size_t kda_paged_tree_decode_workspace_size(int B, int max_nodes, int q_heads, int kv_heads,
                                            int head_dim) {
    if (B < 0 || B > kMaxTreeRequests || max_nodes < 1 || max_nodes > KDA_TREE_MAX_NODES ||
        kv_heads < 1 || q_heads < 1 || (head_dim != 64 && head_dim != 128 && head_dim != 256) ||
        !paged_tree_sizes(B, max_nodes, q_heads, kv_heads, head_dim))
        return 0;
    return kda::paged_tree_workspace_bytes(B, max_nodes, q_heads, kv_heads, head_dim);
}

kda_status kda_paged_tree_decode(const void *q, int64_t q_row_stride, const kda_paged_cache *cache,
                                 const int32_t *block_table, int max_pages,
                                 const int32_t *seq_lens, const int32_t *cu_seqlens,
                                 const uint64_t *ancestors, int B, int64_t N, int max_nodes,
                                 int q_heads, float scale, void *o, float *lse, void *workspace,
                                 size_t workspace_bytes, void *stream) {
    kda::PagedView view;
    kda_status st = paged_view(cache, &view);
    if (st != KDA_OK) return st;
    st = tree_sizes(B, N, max_nodes, B, nullptr);
    if (st != KDA_OK) return st;
    if (max_pages < 0 || q_heads < 1) return KDA_ERR_INVALID_ARG;
    if (!paged_tree_sizes(B, max_nodes, q_heads, view.heads, view.head_dim) ||
        N > INT32_MAX / q_heads)
        return KDA_ERR_UNSUPPORTED_SHAPE;
    const int64_t width = static_cast<int64_t>(q_heads) * view.head_dim;
    if (B > 0 && (seq_lens == nullptr || cu_seqlens == nullptr ||
                  (max_pages > 0 && block_table == nullptr) ||
                  (N > 0 && (q == nullptr || ancestors == nullptr || o == nullptr))))
        return KDA_ERR_INVALID_ARG;
    if (N > 1 && (q_row_stride < width || q_row_stride > INT64_MAX / 4 / N))
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(block_table) || !aligned16(seq_lens) ||
        !aligned16(cu_seqlens) || !aligned16(ancestors) || !aligned16(o) || !aligned16(lse) ||
        !aligned16(workspace) || (N > 1 && q_row_stride % 8 != 0))
        return KDA_ERR_MISALIGNED;
    const size_t need =
        kda::paged_tree_workspace_bytes(B, max_nodes, q_heads, view.heads, view.head_dim);
    if (workspace_bytes < need || (need > 0 && workspace == nullptr))
        return KDA_ERR_WORKSPACE_TOO_SMALL;
    if (B == 0 || N == 0) return KDA_OK;
    const size_t rows = static_cast<size_t>(N) * q_heads, requests = static_cast<size_t>(B) * 4;
    const Buffer outs[] = {{o, rows * view.head_dim * 2}, {lse, rows * 4}, {workspace, need}};
    const Buffer ins[] = {{view.k, view.bytes()}, {view.v, view.bytes()},
                          {view.k_scale, static_cast<size_t>(view.heads) * 4},
                          {view.v_scale, static_cast<size_t>(view.heads) * 4},
                          {block_table, requests * max_pages}, {seq_lens, requests}, {cu_seqlens, requests + 4},
                          {ancestors, static_cast<size_t>(N) * 8}};
    for (int i = 0; i < 3; ++i) {
        if (overlaps_rows(outs[i].p, outs[i].bytes, q, static_cast<size_t>(width) * 2,
                          N > 1 ? static_cast<size_t>(q_row_stride) * 2 : 0, N))
            return KDA_ERR_INVALID_ARG;
        for (const Buffer &in : ins)
            if (overlaps(outs[i].p, outs[i].bytes, in.p, in.bytes)) return KDA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 3; ++j)
            if (overlaps(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return KDA_ERR_INVALID_ARG;
    }
    DeviceInfo *dev = nullptr;
    st = current_device(&dev);
    if (st != KDA_OK) return st;
    kda::TreeAttention a = {};
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.q_row_stride = N > 1 ? q_row_stride : 0;
    a.cache = view;
    a.block_table = block_table;
    a.max_pages = max_pages;
    a.seq_lens = seq_lens;
    a.cu = cu_seqlens;
    a.ancestors = ancestors;
    a.B = B;
    a.q_heads = q_heads;
    a.group = q_heads / view.heads;
    a.max_nodes = max_nodes;
    a.N = N;
    a.scale = scale;
    a.o = static_cast<__nv_bfloat16 *>(o);
    a.lse = lse;
    a.workspace = static_cast<uint8_t *>(workspace);
    a.err = dev->error_word;
    try {
        return from_cuda(kda::launch_paged_tree_decode(a, dev->num_sms,
                                                       static_cast<cudaStream_t>(stream)));
    } catch (...) {  // the list of kernels with raised shared-memory limits could not grow
        return KDA_ERR_CUDA;
    }
}

kda_status kda_paged_compact(const kda_paged_cache *cache, const int32_t *block_table,
                             int max_pages, const int32_t *seq_lens, const int32_t *cu_seqlens,
                             const uint64_t *ancestors, const int32_t *last, int B, int64_t N,
                             int max_nodes, int32_t *kept_lens, void *stream) {
    kda::PagedView view;
    kda_status st = paged_view(cache, &view);
    if (st != KDA_OK) return st;
    st = tree_sizes(B, N, max_nodes, B, nullptr);
    if (st != KDA_OK) return st;
    if (max_pages < 0 || view.k == view.v) return KDA_ERR_INVALID_ARG;
    if (B > 0 && (seq_lens == nullptr || cu_seqlens == nullptr || last == nullptr ||
                  (max_pages > 0 && block_table == nullptr) || (N > 0 && ancestors == nullptr)))
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(block_table) || !aligned16(seq_lens) || !aligned16(cu_seqlens) ||
        !aligned16(ancestors) || !aligned16(last) || !aligned16(kept_lens))
        return KDA_ERR_MISALIGNED;
    const size_t rows = static_cast<size_t>(B) * 4;
    if (overlaps(kept_lens, rows, seq_lens, rows) || overlaps(kept_lens, rows, last, rows) ||
        overlaps(kept_lens, rows, cu_seqlens, rows + 4) ||
        overlaps(kept_lens, rows, ancestors, static_cast<size_t>(N) * 8) ||
        overlaps(kept_lens, rows, block_table, rows * static_cast<size_t>(max_pages)) ||
        overlaps(kept_lens, rows, view.k, view.bytes()) || overlaps(kept_lens, rows, view.v, view.bytes()))
        return KDA_ERR_INVALID_ARG;
    if (B == 0) return KDA_OK;
    DeviceInfo *dev = nullptr;
    st = current_device(&dev);
    if (st != KDA_OK) return st;
    return from_cuda(kda::launch_paged_compact(view, block_table, max_pages, seq_lens, cu_seqlens,
                                               ancestors, last, B, N, max_nodes, kept_lens,
                                               dev->error_word, static_cast<cudaStream_t>(stream)));
}

kda_status kda_page_fork(const int32_t *src, const int32_t *dst, int num_forks, int32_t *seq_lens,
                         const int32_t *free_pages, int num_free, int32_t *block_table,
                         int max_pages, int B, int page_size, int num_pages, int32_t *shares,
                         int32_t *copies, int32_t *pages_used, void *stream) {
    if (num_forks < 0 || num_free < 0 || max_pages < 0 || B < 0 || page_size < 1 || num_pages < 0)
        return KDA_ERR_INVALID_ARG;
    if (static_cast<int64_t>(num_pages) * page_size > INT32_MAX) return KDA_ERR_UNSUPPORTED_SHAPE;
    if (pages_used == nullptr || (num_free > 0 && free_pages == nullptr) ||
        (num_pages > 0 && shares == nullptr) || (B > 0 && seq_lens == nullptr) ||
        (B > 0 && max_pages > 0 && block_table == nullptr) ||
        (num_forks > 0 && (src == nullptr || dst == nullptr || copies == nullptr)))
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(src) || !aligned16(dst) || !aligned16(seq_lens) ||
        (reinterpret_cast<uintptr_t>(free_pages) & 3u) != 0 || !aligned16(block_table) ||
        !aligned16(shares) || !aligned16(copies) || !aligned16(pages_used))
        return KDA_ERR_MISALIGNED;
    const size_t rows = static_cast<size_t>(B) * 4, forks = static_cast<size_t>(num_forks) * 4;
    const struct {
        const void *p;
        size_t bytes;
    } bufs[] = {{seq_lens, rows},
                {block_table, rows * static_cast<size_t>(max_pages)},
                {shares, static_cast<size_t>(num_pages) * 4},
                {copies, forks * 3},
                {pages_used, 4},
                {src, forks},
                {dst, forks},
                {free_pages, static_cast<size_t>(num_free) * 4}};
    for (int i = 0; i < 5; ++i)
        for (int j = i + 1; j < 8; ++j)
            if (overlaps(bufs[i].p, bufs[i].bytes, bufs[j].p, bufs[j].bytes))
                return KDA_ERR_INVALID_ARG;
    DeviceInfo *dev = nullptr;
    kda_status st = current_device(&dev);
    if (st != KDA_OK) return st;
    return from_cuda(kda::launch_page_fork(src, dst, num_forks, seq_lens, free_pages, num_free,
                                           block_table, max_pages, B, page_size, num_pages, shares,
                                           copies, pages_used, dev->error_word,
                                           static_cast<cudaStream_t>(stream)));
}

kda_status kda_paged_copy(const int32_t *copies, int num_copies, const kda_paged_cache *cache,
                          void *stream) {
    kda::PagedView view;
    kda_status st = paged_view(cache, &view);
    if (st != KDA_OK) return st;
    if (num_copies < 0 || view.k == view.v || (num_copies > 0 && copies == nullptr))
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(copies)) return KDA_ERR_MISALIGNED;
    if (num_copies == 0) return KDA_OK;
    DeviceInfo *dev = nullptr;
    st = current_device(&dev);
    if (st != KDA_OK) return st;
    return from_cuda(kda::launch_paged_copy(copies, num_copies, view, dev->error_word,
                                            static_cast<cudaStream_t>(stream)));
}

kda_status kda_page_release(const int32_t *seq_lens, const int32_t *kept_lens,
                            const int32_t *block_table, int max_pages, int B, int page_size,
                            int num_pages, int32_t *shares, int32_t *freed, int max_freed,
                            int32_t *num_freed, void *stream) {
    if (max_pages < 0 || B < 0 || page_size < 1 || num_pages < 0 || max_freed < 0)
        return KDA_ERR_INVALID_ARG;
    if (static_cast<int64_t>(num_pages) * page_size > INT32_MAX ||
        static_cast<int64_t>(B < kda::kReleaseRequests ? B : kda::kReleaseRequests) * max_pages > INT32_MAX)
        return KDA_ERR_UNSUPPORTED_SHAPE;
    if (num_freed == nullptr || (max_freed > 0 && freed == nullptr) ||
        (num_pages > 0 && shares == nullptr) ||
        (B > 0 && (seq_lens == nullptr || kept_lens == nullptr ||
                   (max_pages > 0 && block_table == nullptr))))
        return KDA_ERR_INVALID_ARG;
    if (!aligned16(seq_lens) || !aligned16(kept_lens) || !aligned16(block_table) ||
        !aligned16(shares) || (reinterpret_cast<uintptr_t>(freed) & 3u) != 0 ||
        !aligned16(num_freed))
        return KDA_ERR_MISALIGNED;
    const size_t rows = static_cast<size_t>(B) * 4;
    const struct {
        const void *p;
        size_t bytes;
    } bufs[] = {{shares, static_cast<size_t>(num_pages) * 4},
                {freed, static_cast<size_t>(max_freed) * 4},
                {num_freed, 4},
                {seq_lens, rows},
                {kept_lens, rows},
                {block_table, rows * static_cast<size_t>(max_pages)}};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 6; ++j)
            if (overlaps(bufs[i].p, bufs[i].bytes, bufs[j].p, bufs[j].bytes))
                return KDA_ERR_INVALID_ARG;
    DeviceInfo *dev = nullptr;
    kda_status st = current_device(&dev);
    if (st != KDA_OK) return st;
    try {
        return from_cuda(kda::launch_page_release(seq_lens, kept_lens, block_table, max_pages, B,
                                                  page_size, num_pages, shares, freed, max_freed,
                                                  num_freed, dev->error_word,
                                                  static_cast<cudaStream_t>(stream)));
    } catch (...) {  // the list of kernels with raised shared-memory limits could not grow
        return KDA_ERR_CUDA;
    }
}

kda_status kda_debug_check_gate_division(uint64_t *mismatches, void *stream) {
    if (mismatches == nullptr) return KDA_ERR_INVALID_ARG;
    DeviceInfo *dev = nullptr;
    kda_status st = current_device(&dev);
    if (st != KDA_OK) return st;
    unsigned long long n = 0;
    st = from_cuda(kda::check_gate_division(&n, dev->num_sms, static_cast<cudaStream_t>(stream)));
    if (st != KDA_OK) return st;
    *mismatches = static_cast<uint64_t>(n);
    return KDA_OK;
}

kda_status kda_debug_set_wait_limit(int64_t copy_polls, int64_t product_polls) {
    kda::set_prefill_wait_polls(copy_polls, product_polls);
    return KDA_OK;
}

kda_status kda_get_last_device_error(void *stream) {
    DeviceInfo *dev = nullptr;
    kda_status st = current_device(&dev);
    if (st != KDA_OK) return st;
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return KDA_ERR_CUDA;
    }
    unsigned int word = 0;
    if (cudaMemcpyFromSymbol(&word, g_device_error_word, sizeof(word)) != cudaSuccess) {
        cudaGetLastError();
        return KDA_ERR_CUDA;
    }
    if (word != 0) {
        const unsigned int zero = 0;
        if (cudaMemcpyToSymbol(g_device_error_word, &zero, sizeof(zero)) != cudaSuccess) {
            cudaGetLastError();
            return KDA_ERR_CUDA;
        }
    }
    return static_cast<kda_status>(word);
}

}  // extern "C"
