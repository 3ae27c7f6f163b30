// verify.cuh -- parameters of the kernel that verifies drafted token trees
// (verify.cu), filled in ops_pages.cu.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace b2pa {

// Nodes of a request at most: six words each in shared memory.
constexpr int kVerifyMaxNodes = 4096;

struct VerifyParams {
    const float* target;  // [T, V]
    const float* draft;   // [T, V] or null
    long long target_st, draft_st;
    const int *tokens, *parents;       // [T]
    const float *uniforms, *last;      // [T], [B]
    const int* cum_q;                  // [B + 1]
    int* accepted;                     // [B, width]
    long long acc_st;
    int *counts, *next;                // [B]
    unsigned* err;
    int B, T, V, max_q, width;
    int aligned;  // rows can be read in 16-byte pieces
};

cudaError_t launch_verify(const VerifyParams& p, int sms, cudaStream_t stream);

}  // namespace b2pa
