// kda_paged_tree_d256.cu -- tree attention: 256 channels.
#include "kda_paged_tree.cuh"

namespace kda {
namespace treeatt {

template cudaError_t launch_dim<256>(const Args &, int, int, cudaStream_t);

}  // namespace treeatt
}  // namespace kda
