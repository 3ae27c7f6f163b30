// rope.cuh -- parameters of the query/key norm and rotation kernel (rope.cu),
// filled by b2pa_qk_norm_rope in ops.cu.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace b2pa {

constexpr int kRopeMaxD = 256;
constexpr int kRopeMaxAxes = 4;

struct RopeTensor {
    const uint16_t* in;  // bf16 [T, heads, D], head_dim contiguous
    uint16_t* out;
    long long in_tok, in_head, out_tok, out_head;  // element strides
    const void* weight;                            // [D] bf16 or fp32, or null: no norm
    int weight_f32;
    int heads;
};

struct RopeParams {
    RopeTensor x[2];         // queries, keys
    const float* cos_sin;    // [max_pos, R]: R / 2 cosines, then R / 2 sines
    long long cs_stride;
    const int* positions;    // [axes, T]
    long long pos_stride;    // between axes
    int T, D, R, axes, max_pos;
    int vec_table;           // 1: four consecutive table entries can be read as one float4
    float eps;
    float inv_d;             // 1 / D
    unsigned* err;
    uint8_t axis_of[kRopeMaxD / 2];  // axis of each frequency
    // per four frequencies: their common axis, or 255
    uint8_t axis_of4[kRopeMaxD / 8];
};

// interleaved: element pairs (2i, 2i + 1) rotate; else (i, i + R / 2)
cudaError_t launch_qk_norm_rope(const RopeParams& p, bool interleaved, int sms, cudaStream_t stream);

}  // namespace b2pa
