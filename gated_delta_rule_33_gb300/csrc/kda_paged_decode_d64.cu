// kda_paged_decode_d64.cu -- the one-token attention's kernels for 64 channels.
#include "kda_paged_decode.cuh"

namespace kda {
namespace paged {
template cudaError_t launch_paged_decode_dim<64>(const Args &, bool, int, int, cudaStream_t);
}  // namespace paged
}  // namespace kda
