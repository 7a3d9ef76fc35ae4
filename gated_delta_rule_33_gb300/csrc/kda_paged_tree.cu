// kda_paged_tree.cu -- tree attention: 128 channels, and the choice of a kernel.
#include "kda_paged_tree.cuh"

namespace kda {
namespace treeatt {

template <int kD>
cudaError_t launch_dim(const Args &a, int m, int ctas, cudaStream_t s);
extern template cudaError_t launch_dim<64>(const Args &, int, int, cudaStream_t);
extern template cudaError_t launch_dim<256>(const Args &, int, int, cudaStream_t);

}  // namespace treeatt

size_t paged_tree_workspace_bytes(int B, int max_nodes, int q_heads, int kv_heads, int head_dim) {
    if (B == 0) return 0;
    return 2 * treeatt::kMaxCtas *
           treeatt::slot_bytes(treeatt::m_tiles(max_nodes, q_heads / kv_heads, head_dim), head_dim);
}

cudaError_t launch_paged_tree_decode(const TreeAttention &t, int num_sms, cudaStream_t s) {
    const int ctas = num_sms < treeatt::kMaxCtas ? num_sms : treeatt::kMaxCtas;
    const int m = treeatt::m_tiles(t.max_nodes, t.group, t.cache.head_dim);
    treeatt::Args a = {};
    a.t = t;
    a.group = FastDiv(static_cast<uint32_t>(t.group));
    a.cut = reinterpret_cast<float *>(t.workspace);
    a.ml = a.cut + static_cast<size_t>(2) * treeatt::kMaxCtas * m * 128 * t.cache.head_dim;
    switch (t.cache.head_dim) {
        case 64: return treeatt::launch_dim<64>(a, m, ctas, s);
        case 128: return treeatt::launch_dim<128>(a, m, ctas, s);
        default: return treeatt::launch_dim<256>(a, m, ctas, s);
    }
}

}  // namespace kda
