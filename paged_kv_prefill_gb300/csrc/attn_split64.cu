// attn_split64.cu -- instantiations of attn_split.cuh for bf16 caches, head_dim 64
#include "attn_split_impl.cuh"

namespace b2pa {

template cudaError_t launch_split<64, false, 2, 0>(const TreeParams&, cudaStream_t);
template cudaError_t launch_split<64, false, 1, 1>(const TreeParams&, cudaStream_t);
template cudaError_t launch_split<64, false, 1, 2>(const TreeParams&, cudaStream_t);
template cudaError_t launch_split<64, false, 2, 1>(const TreeParams&, cudaStream_t);
template cudaError_t launch_split<64, false, 2, 2>(const TreeParams&, cudaStream_t);

}  // namespace b2pa
