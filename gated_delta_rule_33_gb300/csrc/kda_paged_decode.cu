// kda_paged_decode.cu -- the launcher of the one-token attention over a paged
// cache (kernels: kda_paged_decode.cuh), and its kernels for 128 channels.
#include "kda_paged_decode.cuh"

namespace kda {
namespace paged {
extern template cudaError_t launch_paged_decode_dim<64>(const Args &, bool, int, int, cudaStream_t);
extern template cudaError_t launch_paged_decode_dim<256>(const Args &, bool, int, int, cudaStream_t);
}  // namespace paged

size_t paged_decode_workspace_bytes(int, int q_heads, int kv_heads, int head_dim) {
    return paged::layout_bytes(paged::unit_heads(q_heads / kv_heads, head_dim), head_dim, nullptr, nullptr);
}

cudaError_t launch_paged_decode(const __nv_bfloat16 *q, int64_t q_row_stride,
                                const PagedView &cache, const int32_t *block_table, int max_pages,
                                const int32_t *seq_lens, int B, int q_heads, float scale, void *o,
                                bool o_bf16, float *lse, void *workspace, unsigned int *err,
                                int num_sms, cudaStream_t s) {
    paged::Args a;
    a.q = q;
    a.q_row_stride = q_row_stride;
    a.cache = cache;
    a.block_table = block_table;
    a.max_pages = max_pages;
    a.seq_lens = seq_lens;
    a.B = B;
    a.q_heads = q_heads;
    a.group = q_heads / cache.heads;
    const int heads = paged::unit_heads(a.group, cache.head_dim);
    a.head_tiles = (a.group + heads - 1) / heads;
    a.scale = scale;
    a.o = o;
    a.lse = lse;
    a.err = err;
    paged::layout_bytes(heads, cache.head_dim, static_cast<uint8_t *>(workspace), &a.ws);
    const int ctas = num_sms < paged::kMaxCtas ? num_sms : paged::kMaxCtas;
    const auto launch = cache.head_dim == 64    ? paged::launch_paged_decode_dim<64>
                        : cache.head_dim == 128 ? paged::launch_paged_decode_dim<128>
                                                : paged::launch_paged_decode_dim<256>;
    return launch(a, o_bf16, heads, ctas, s);
}

}  // namespace kda
