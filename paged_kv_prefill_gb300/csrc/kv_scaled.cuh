// kv_scaled.cuh -- parameters of the kernels that write and read an e4m3 cache
// with one scale per (token, kv head) row (kv_scaled.cu), filled in ops.cu.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace b2pa {

// Index 0: K, 1: V.  Pool and scale strides by (page, kv head, slot), elements.
struct ScaledKvParams {
    const uint16_t* x[2];  // write: bf16 [T, Hkv, D]
    uint16_t* y[2];        // read: bf16 [T, Hkv, D]
    long long tok[2], head[2];  // element strides of x or y (head_dim contiguous)
    uint8_t* pool[2];      // e4m3
    long long pool_st[2][3];
    float* scale[2];
    long long scale_st[2][3];
    const int* cache_loc;  // [T]: page * page_size + slot
    int T, Hkv, D, page_size, num_pages;
    unsigned* err;
};

cudaError_t launch_append_scaled(const ScaledKvParams& p, cudaStream_t stream);
cudaError_t launch_read_scaled(const ScaledKvParams& p, cudaStream_t stream);

}  // namespace b2pa
