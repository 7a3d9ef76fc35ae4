// kda_paged_decode.cu -- softmax attention of one new token per sequence over a
// paged key-value cache.
//
//   s_j = scale <q, k_j>,  m = max_j s_j,  l = sum_j e^{s_j - m}
//   o = sum_j e^{s_j - m} v_j / l,  lse = m + log l
//
// One CTA per (sequence, query head): warp w walks keys w, w + 8, ... with a
// running maximum and sum, and the warps' results are joined in shared memory:
// m = max m_w, o = sum e^{m_w - m} o_w / sum e^{m_w - m} l_w.
#include <cuda_fp8.h>

#include "kda_internal.cuh"
#include "kda_paged.cuh"

namespace kda {
namespace {

constexpr int kWarps = 8;

template <bool kFp8>
__device__ __forceinline__ float cache_value(const uint8_t *p, int d) {
    if constexpr (kFp8) {
        __nv_fp8_e4m3 x;
        x.__x = p[d];
        return static_cast<float>(x);
    } else {
        return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[d]);
    }
}

template <int kD, bool kFp8>
__global__ void __launch_bounds__(kWarps * 32) paged_decode_kernel(
    const __nv_bfloat16 *__restrict__ q, int64_t q_row_stride, const PagedView cache,
    const int32_t *__restrict__ block_table, int max_pages, const int32_t *__restrict__ seq_lens,
    int q_heads, float scale, void *__restrict__ o, bool o_bf16, float *__restrict__ lse,
    unsigned int *err) {
    constexpr int kPer = kD / 32;
    __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][kD];
    const int64_t row = blockIdx.x;
    const int b = static_cast<int>(row / q_heads), hq = static_cast<int>(row % q_heads);
    const int h = hq / (q_heads / cache.heads);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int len = seq_lens[b];
    if (len < 0 || len > static_cast<int64_t>(max_pages) * cache.page.d) {
        if (threadIdx.x == 0) record_device_error(err, kDevInvalidArg);
        len = 0;
    }
    float qv[kPer], acc[kPer];
    const float ks = cache.k_scale == nullptr ? 1.f : cache.k_scale[h];
    const float vs = cache.v_scale == nullptr ? 1.f : cache.v_scale[h];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        qv[i] = __bfloat162float(q[b * q_row_stride + hq * kD + lane + 32 * i]);
        acc[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int j = warp; j < len; j += kWarps) {
        uint32_t idx, r;
        cache.page.divmod(j, idx, r);
        const int p = block_table[static_cast<int64_t>(b) * max_pages + idx];
        if (p < 0 || p >= cache.num_pages) {
            if (lane == 0) record_device_error(err, kDevInvalidArg);
            continue;
        }
        const int64_t at = p * cache.page_stride + r * cache.token_stride + h * cache.head_stride;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            s = fmaf(qv[i], cache_value<kFp8>(cache.k + at, lane + 32 * i), s);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= scale * ks;
        const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn;
        const float f = expf(m - ref), e = expf(s - ref);
        l = l * f + e;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            acc[i] = fmaf(e, cache_value<kFp8>(cache.v + at, lane + 32 * i), acc[i] * f);
        m = mn;
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) s_o[warp][lane + 32 * i] = acc[i];
    __syncthreads();
    float mm = -INFINITY, ll = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w]);
    const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) ll += expf(s_m[w] - ref) * s_l[w];
    if (threadIdx.x < kD) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) x += expf(s_m[w] - ref) * s_o[w][threadIdx.x];
        x = ll == 0.f ? 0.f : x / ll * vs;
        if (o_bf16)
            static_cast<__nv_bfloat16 *>(o)[row * kD + threadIdx.x] = __float2bfloat16_rn(x);
        else
            static_cast<float *>(o)[row * kD + threadIdx.x] = x;
    }
    if (threadIdx.x == 0 && lse != nullptr) lse[row] = ll == 0.f ? -INFINITY : mm + logf(ll);
}

template <int kD>
cudaError_t launch_dim(const __nv_bfloat16 *q, int64_t q_row_stride, const PagedView &cache,
                       const int32_t *block_table, int max_pages, const int32_t *seq_lens, int B,
                       int q_heads, float scale, void *o, bool o_bf16, float *lse,
                       unsigned int *err, cudaStream_t s) {
    const unsigned rows = static_cast<unsigned>(B) * q_heads;
    auto kern = cache.fp8 ? paged_decode_kernel<kD, true> : paged_decode_kernel<kD, false>;
    kern<<<rows, kWarps * 32, 0, s>>>(q, q_row_stride, cache, block_table, max_pages, seq_lens,
                                      q_heads, scale, o, o_bf16, lse, err);
    return cudaGetLastError();
}

}  // namespace

size_t paged_decode_workspace_bytes(int, int, int, int) { return 16; }

cudaError_t launch_paged_decode(const __nv_bfloat16 *q, int64_t q_row_stride,
                                const PagedView &cache, const int32_t *block_table, int max_pages,
                                const int32_t *seq_lens, int B, int q_heads, float scale, void *o,
                                bool o_bf16, float *lse, void *, unsigned int *err, int,
                                cudaStream_t s) {
    auto launch = cache.head_dim == 64    ? launch_dim<64>
                  : cache.head_dim == 128 ? launch_dim<128>
                                          : launch_dim<256>;
    return launch(q, q_row_stride, cache, block_table, max_pages, seq_lens, B, q_heads, scale, o,
                  o_bf16, lse, err, s);
}

}  // namespace kda
