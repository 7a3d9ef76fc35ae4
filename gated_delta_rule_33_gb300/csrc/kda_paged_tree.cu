// kda_paged_tree.cu -- softmax attention of a tree of drafted tokens per sequence over a paged
// key-value cache that holds the drafted tokens' keys and values too.
//
// Node i of a sequence with L keys, n of them drafted, sees the C = L - n keys of the context
// and the drafted key j (at position C + j) where bit j of its word is set:
//
//   s_j = scale <q_i, k_j>,  m = max_j s_j,  l = sum_j e^{s_j - m}
//   o = sum_j e^{s_j - m} v_j / l,  lse = m + log l
//
// over the keys j that it sees; a node that sees none has o = 0 and lse = -inf.
#include <cuda_fp16.h>

#include "kda_tree.cuh"

namespace kda {
namespace {

constexpr int kWarps = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// A lane's kN neighbouring values of a row, widened.
template <bool kFp8, int kN>
__device__ __forceinline__ void load_values(const uint8_t *p, float (&x)[kN]) {
#pragma unroll
    for (int i = 0; i < kN; i += 2) {
        if constexpr (kFp8) {
            uint32_t y;
            const uint16_t raw = *reinterpret_cast<const uint16_t *>(p + i);
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"(raw));
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&y));
            x[i] = f.x;
            x[i + 1] = f.y;
        } else {
            const uint32_t raw = *reinterpret_cast<const uint32_t *>(p + 2 * i);
            x[i] = __uint_as_float(raw << 16);
            x[i + 1] = __uint_as_float(raw & 0xffff0000u);
        }
    }
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// One warp a (node, query head).
template <int kD, bool kFp8>
__global__ void __launch_bounds__(kWarps * 32) tree_attention_kernel(const TreeAttention a) {
    constexpr int kN = kD / 32;
    wait_for_kernel_before();
    const int lane = threadIdx.x & 31, b = blockIdx.y;
    const TreeRows t = tree_rows(a.cu, b, a.N, a.max_nodes);
    const int len = a.seq_lens[b];
    const bool fits = len >= t.rows && len <= static_cast<int64_t>(a.max_pages) * a.cache.page.d;
    if ((t.bad || !fits) && threadIdx.x == 0) record_device_error(a.err, kDevInvalidArg);
    const int64_t rows = static_cast<int64_t>(t.rows) * a.q_heads;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); r < rows;
         r += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t row = t.first + r / a.q_heads;
        const int qh = static_cast<int>(r % a.q_heads), h = qh / a.group;
        const int keys = fits && t.n > 0 ? len : 0, context = len - t.n;
        const uint64_t word = a.ancestors[row];
        float q[kN], acc[kN], m = -INFINITY, l = 0.f;
        load_values<false, kN>(reinterpret_cast<const uint8_t *>(a.q + row * a.q_row_stride +
                                                                 qh * kD + lane * kN),
                               q);
        const float c = a.scale * kLog2e * (a.cache.k_scale != nullptr ? a.cache.k_scale[h] : 1.f);
#pragma unroll
        for (int i = 0; i < kN; ++i) acc[i] = 0.f;
        for (int j = 0; j < keys; ++j) {
            if (j >= context && !((word >> (j - context)) & 1)) continue;
            uint32_t idx, in_page;
            a.cache.page.divmod(j, idx, in_page);
            const int page = a.block_table[static_cast<int64_t>(b) * a.max_pages + idx];
            if (page < 0 || page >= a.cache.num_pages) {
                if (lane == 0) record_device_error(a.err, kDevInvalidArg);
                continue;
            }
            const int64_t off = page * a.cache.page_stride + in_page * a.cache.token_stride +
                                h * a.cache.head_stride + lane * kN * (kFp8 ? 1 : 2);
            float k[kN], v[kN], s = 0.f;
            load_values<kFp8, kN>(a.cache.k + off, k);
            load_values<kFp8, kN>(a.cache.v + off, v);
#pragma unroll
            for (int i = 0; i < kN; ++i) s += q[i] * k[i];
            s = warp_sum(s) * c;
            const float to = s > m || s != s ? s : m;
            const float from = to == -INFINITY ? 0.f : to;
            const float keep = exp2f(m - from), p = exp2f(s - from);
            m = to;
            const float before = l * keep;
            l = before + p;
            if (l == 0.f) continue;
            // an average from the first key on: as large as the values, not as their sum
            const float w = p / l, rest = before / l;
#pragma unroll
            for (int i = 0; i < kN; ++i) acc[i] = acc[i] * rest + w * v[i];
        }
        const float vs = a.cache.v_scale != nullptr ? a.cache.v_scale[h] : 1.f;
        const int64_t out = row * a.q_heads + qh;
#pragma unroll
        for (int i = 0; i < kN; ++i)
            a.o[out * kD + lane * kN + i] = __float2bfloat16_rn(l == 0.f ? 0.f : acc[i] * vs);
        if (a.lse != nullptr && lane == 0) a.lse[out] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
}

}  // namespace

size_t paged_tree_workspace_bytes(int B, int max_nodes, int q_heads, int kv_heads, int head_dim) {
    return B > 0 ? 16 : 0;
}

cudaError_t launch_paged_tree_decode(const TreeAttention &a, int num_sms, cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(a.max_nodes) * a.q_heads;
    const dim3 grid(static_cast<unsigned>((rows + kWarps - 1) / kWarps), a.B);
    auto run = [&](auto kernel) { return launch_early(kernel, grid, kWarps * 32, 0, s, a); };
    const bool fp8 = a.cache.fp8;
    switch (a.cache.head_dim) {
        case 64: return run(fp8 ? tree_attention_kernel<64, true> : tree_attention_kernel<64, false>);
        case 128: return run(fp8 ? tree_attention_kernel<128, true> : tree_attention_kernel<128, false>);
        default: return run(fp8 ? tree_attention_kernel<256, true> : tree_attention_kernel<256, false>);
    }
}

}  // namespace kda
