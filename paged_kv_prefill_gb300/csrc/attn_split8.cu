// attn_split8.cu -- instantiations of attn_split.cuh for e4m3 caches
#include "attn_split_impl.cuh"

namespace b2pa {

template cudaError_t launch_split<128, true, 2, 0>(const TreeParams&, cudaStream_t);
template cudaError_t launch_split<128, true, 1, 1>(const TreeParams&, cudaStream_t);
template cudaError_t launch_split<128, true, 1, 2>(const TreeParams&, cudaStream_t);
template cudaError_t launch_split<128, true, 2, 1>(const TreeParams&, cudaStream_t);
template cudaError_t launch_split<128, true, 2, 2>(const TreeParams&, cudaStream_t);

}  // namespace b2pa
