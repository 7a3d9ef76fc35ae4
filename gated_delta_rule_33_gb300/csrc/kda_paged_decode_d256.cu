// kda_paged_decode_d256.cu -- the one-token attention's kernels for 256 channels.
#include "kda_paged_decode.cuh"

namespace kda {
namespace paged {
template cudaError_t launch_paged_decode_dim<256>(const Args &, bool, int, int, cudaStream_t);
}  // namespace paged
}  // namespace kda
