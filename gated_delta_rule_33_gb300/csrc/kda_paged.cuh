// kda_paged.cuh -- the paged key-value cache as the kernels see it, and the
// launchers of its three entry points (kda_page_plan, kda_paged_append,
// kda_paged_decode).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace kda {

// Division of 0 <= n < 2^31 by a fixed d >= 1 as a multiply-high, an add and a
// shift.  With l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1,
// floor(n / d) = (floor(m n / 2^32) + n) >> l  (Granlund and Montgomery,
// "Division by invariant integers using multiplication", 1994, theorem 4.2).
struct FastDiv {
    uint32_t d, mul, shift;

    FastDiv() = default;
    explicit FastDiv(uint32_t div) : d(div), shift(0) {
        while ((uint64_t{1} << shift) < d) ++shift;
        mul = static_cast<uint32_t>((((uint64_t{1} << shift) - d) << 32) / d + 1);
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const {
        return (__umulhi(mul, n) + n) >> shift;
    }
    __device__ __forceinline__ void divmod(uint32_t n, uint32_t &q, uint32_t &r) const {
        q = div(n);
        r = n - q * d;
    }
};

// The paged kernels are launched so that their blocks may be set up while the kernel
// before them ends (programmatic dependent launch): they wait for that kernel, all of
// it, before they touch memory, and only then let the next one be set up.
//
// What they read after the wait may have been written while they were being set up, so
// it is read by ordinary loads: not by __ldg or through __restrict__, which promise that
// the data stays as it is for as long as the kernel lives and which nothing keeps below
// the wait.
__device__ __forceinline__ void wait_for_kernel_before() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// An ordinary 16-byte load whose data is not wanted again.
__device__ __forceinline__ uint4 load_once(const uint4 *p) {
    uint4 x;
    asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                 : "l"(p));
    return x;
}

template <class... Params, class... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int threads, size_t smem,
                         cudaStream_t s, const Args &...args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// One layer's cache.  Strides are in bytes.
struct PagedView {
    uint8_t *k, *v;
    const float *k_scale, *v_scale;  // [heads] or null
    int64_t page_stride, token_stride, head_stride;
    FastDiv page;                    // by page_size
    int num_pages;
    int heads, head_dim;
    bool fp8;
};

cudaError_t launch_page_plan(const int32_t *cached_lens, const int32_t *new_lens,
                             const int32_t *free_pages, int num_free, int32_t *block_table,
                             int max_pages, int B, int page_size, int num_pages,
                             int32_t *seq_lens, int32_t *cu_seqlens, int32_t *slot_map, int64_t N,
                             int32_t *pages_used, unsigned int *err, cudaStream_t s);

cudaError_t launch_paged_append(const __nv_bfloat16 *k, const __nv_bfloat16 *v,
                                int64_t k_row_stride, int64_t v_row_stride,
                                const int32_t *slot_map, int64_t N, const PagedView &cache,
                                unsigned int *err, cudaStream_t s);

size_t paged_decode_workspace_bytes(int B, int q_heads, int kv_heads, int head_dim);

cudaError_t launch_paged_decode(const __nv_bfloat16 *q, int64_t q_row_stride,
                                const PagedView &cache, const int32_t *block_table, int max_pages,
                                const int32_t *seq_lens, int B, int q_heads, float scale, void *o,
                                bool o_bf16, float *lse, void *workspace, unsigned int *err,
                                int num_sms, cudaStream_t s);

}  // namespace kda
