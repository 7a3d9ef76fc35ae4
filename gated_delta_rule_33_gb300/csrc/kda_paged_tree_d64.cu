// kda_paged_tree_d64.cu -- tree attention: 64 channels.
#include "kda_paged_tree.cuh"

namespace kda {
namespace treeatt {

template cudaError_t launch_dim<64>(const Args &, int, int, cudaStream_t);

}  // namespace treeatt
}  // namespace kda
