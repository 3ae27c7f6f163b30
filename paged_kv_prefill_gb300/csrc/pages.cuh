// pages.cuh -- parameters of the kernels that move rows and whole pages of the
// pools and keep the page ledger (pages.cu), filled in ops_pages.cu.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace b2pa {

// One tensor of a cache (K, V, or one's scales), in bytes.
struct Plane {
    uint8_t* base;
    long long st[3];  // page, kv head, slot
    int row;          // bytes of a row
    int vec;          // bytes of a piece: the largest of 16, 8, 4, 2, 1 that divides addresses, strides and rows
};
constexpr int kMaxPlanes = 4;

struct CopyPagesParams {
    Plane plane[kMaxPlanes];
    // how a page of each plane is gone through: `outer` x `inner` rows of `row`
    // bytes (1 x 1 where the page lies in one piece)
    int outer[kMaxPlanes], inner[kMaxPlanes];
    long long outer_st[kMaxPlanes], inner_st[kMaxPlanes], row[kMaxPlanes];
    int blocks[kMaxPlanes];  // per page
    int planes, n, num_pages;
    const int *src, *dst;
    unsigned* err;
};

struct CompactParams {
    Plane plane[kMaxPlanes];
    int planes, pieces;  // pieces of a token over all planes
    int Hkv, page_size, num_pages, max_pages;
    const int* block_tables;
    long long bt_stride;
    const int *seq_lens, *cum_q, *counts;
    const int* accepted;
    long long acc_stride;
    int width;  // columns of accepted
    int* new_lens;
    unsigned* err;
    int B;
};

// Requests of one fork or grow call: each keeps four words in shared memory (grow: uses three).
constexpr int kLedgerMax = 4096;

struct LedgerParams {
    int* tables;  // [R, max_pages]
    long long stride;
    int* seq;     // [R]
    int* refs;    // [N]
    const int *rows, *parents, *to;  // [n]: children or rows; fork's parents; grow's new lengths
    int *src, *dst;                  // [n], fork
    unsigned* err;
    int n, R, max_pages, N, page_size;
};

cudaError_t launch_copy_pages(const CopyPagesParams& p, cudaStream_t stream);
cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream);
cudaError_t launch_free_pages(const LedgerParams& p, cudaStream_t stream);
cudaError_t launch_take_pages(const LedgerParams& p, bool fork, cudaStream_t stream);

}  // namespace b2pa
