// kda_paged_append.cu -- new keys and values into a paged cache, by slot.
//
//   cache[slot / page_size, slot % page_size, h, :] = x[n, h, :]
//   (8-bit: e4m3(x / scale[h]), the fp32 quotient rounded to nearest)
//
// A copy: HBM-bound, 4 (or 3) bytes moved per value.  A thread moves 16-byte
// pieces of the flattened [token, head, channel] rows; neighbouring threads move
// neighbouring pieces, so that both sides are whole 32-byte sectors in any
// layout.  Two pieces to a thread overlap their loads (16384 tokens of 8 heads of
// 128, bf16: 21.5 us, 92 % of HBM; 23.3 with one, 21.6 with four); an 8-bit piece
// is two loads already (9001 tokens of 4 heads of 256: 10.2 us with one, 11.0
// with two).  Both sides are streamed past L2's other contents.
#include <cuda_fp8.h>

#include "kda_internal.cuh"
#include "kda_paged.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
template <bool kFp8>
constexpr int kUnits = kFp8 ? 1 : 2;

// x / y, y a positive normal scale with reciprocal r: one correction with the
// exact remainder rounds the quotient correctly (Markstein, IBM J. Res. Dev.
// 34(1), 1990) where nothing under- or overflows; the remainder of an infinite
// or NaN quotient is left out.
__device__ __forceinline__ float quotient(float x, float y, float r) {
    const float q = x * r;
    const float e = __fmaf_rn(-q, y, x);
    return fabsf(q) < 1e30f ? __fmaf_rn(e, r, q) : q;
}

__device__ __forceinline__ uint32_t to_e4m3x4(const uint32_t lo, const uint32_t hi, float y,
                                              float r) {
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&lo));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&hi));
    const uint32_t u = __nv_cvt_float2_to_fp8x2(
        make_float2(quotient(a.x, y, r), quotient(a.y, y, r)), __NV_SATFINITE, __NV_E4M3);
    const uint32_t w = __nv_cvt_float2_to_fp8x2(
        make_float2(quotient(b.x, y, r), quotient(b.y, y, r)), __NV_SATFINITE, __NV_E4M3);
    return u | (w << 16);
}

// blockIdx.y: 0 keys, 1 values.  A unit is 8 source values (16 for an 8-bit
// cache): 16 bytes of the cache.
template <bool kFp8>
__global__ void __launch_bounds__(kThreads) append_kernel(
    const __nv_bfloat16 *k, const __nv_bfloat16 *v, int64_t k_row_stride,
    int64_t v_row_stride, const int32_t *slot_map, int64_t N, const PagedView cache,
    FastDiv row, int dim_shift, unsigned int *err) {
    constexpr int kVals = kFp8 ? 16 : 8;
    wait_for_kernel_before();
    const bool is_v = blockIdx.y != 0;
    const __nv_bfloat16 *x = is_v ? v : k;
    const int64_t x_stride = is_v ? v_row_stride : k_row_stride;
    uint8_t *dst = is_v ? cache.v : cache.k;
    const float *scales = is_v ? cache.v_scale : cache.k_scale;

    const int64_t u0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kUnits<kFp8>);
    const int64_t n0 = u0 / row.d;
    const uint32_t r0 = static_cast<uint32_t>(u0 - n0 * row.d);

    uint4 val[kUnits<kFp8>][kFp8 ? 2 : 1];
    int slot[kUnits<kFp8>];
    int head[kUnits<kFp8>], dim[kUnits<kFp8>];
#pragma unroll
    for (int i = 0; i < kUnits<kFp8>; ++i) {
        uint32_t dn, u;
        row.divmod(r0 + threadIdx.x + i * kThreads, dn, u);
        const int64_t n = n0 + dn;
        slot[i] = -1;
        if (n < N) {
            slot[i] = slot_map[n];
            const int flat = static_cast<int>(u) * kVals;
            head[i] = flat >> dim_shift;
            dim[i] = flat - (head[i] << dim_shift);
            const uint4 *src = reinterpret_cast<const uint4 *>(x + n * x_stride + flat);
            val[i][0] = load_once(src);
            if constexpr (kFp8) val[i][1] = load_once(src + 1);
        }
    }
#pragma unroll
    for (int i = 0; i < kUnits<kFp8>; ++i) {
        if (slot[i] < 0) continue;
        uint32_t p, r;
        cache.page.divmod(static_cast<uint32_t>(slot[i]), p, r);
        if (p >= static_cast<uint32_t>(cache.num_pages)) {
            record_device_error(err, kDevInvalidArg);
            continue;
        }
        uint8_t *to = dst + p * cache.page_stride + r * cache.token_stride +
                      head[i] * cache.head_stride + dim[i] * (kFp8 ? 1 : 2);
        uint4 out;
        if constexpr (kFp8) {
            const float y = scales == nullptr ? 1.f : scales[head[i]];
            const float rcp = __frcp_rn(y);
            out.x = to_e4m3x4(val[i][0].x, val[i][0].y, y, rcp);
            out.y = to_e4m3x4(val[i][0].z, val[i][0].w, y, rcp);
            out.z = to_e4m3x4(val[i][1].x, val[i][1].y, y, rcp);
            out.w = to_e4m3x4(val[i][1].z, val[i][1].w, y, rcp);
        } else {
            out = val[i][0];
        }
        __stcs(reinterpret_cast<uint4 *>(to), out);
    }
}

}  // namespace

cudaError_t launch_paged_append(const __nv_bfloat16 *k, const __nv_bfloat16 *v,
                                int64_t k_row_stride, int64_t v_row_stride,
                                const int32_t *slot_map, int64_t N, const PagedView &cache,
                                unsigned int *err, cudaStream_t s) {
    const uint32_t units = static_cast<uint32_t>(cache.heads) * cache.head_dim / (cache.fp8 ? 16 : 8);
    const int per_cta = kThreads * (cache.fp8 ? kUnits<true> : kUnits<false>);
    const int64_t ctas = (N * units + per_cta - 1) / per_cta;
    int dim_shift = 0;
    while ((1 << dim_shift) < cache.head_dim) ++dim_shift;
    const dim3 grid(static_cast<unsigned>(ctas), 2);
    const FastDiv row(units);
    return launch_early(cache.fp8 ? append_kernel<true> : append_kernel<false>, grid, kThreads, 0, s,
                        k, v, k_row_stride, v_row_stride, slot_map, N, cache, row, dim_shift, err);
}

}  // namespace kda
