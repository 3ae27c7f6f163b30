// host.cuh -- host-side helpers that the entry points of b2pa.cu and ops.cu
// share: errors, device properties, status words, argument checks and tensor
// maps.  Defined in b2pa.cu where nothing else is said.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/b2pa.h"

namespace b2pa {

// Set the thread's error text and return `status`.
int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int cuda_fail(cudaError_t e, const char* what);
void clear_error();

// No C++ exception (an allocation that failed) may leave a C entry point.
template <typename F>
int guarded(F&& f)
{
    try {
        clear_error();
        return f();
    } catch (...) {
        return B2PA_ERR_CUDA;
    }
}

// the process-wide options
int kernel_path();
unsigned long long wait_limit_ns();
int inject_stall();

struct DevInfo {
    bool init = false;
    int sms = 0;
    int major = 0, minor = 0;
};
int device_info(int* dev_out, DevInfo* info);

// The device error word of (device, stream) for an entry point that keeps no
// workspace: at one address until b2pa_release.
int status_word(int dev, cudaStream_t stream, unsigned** out);

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();

bool is_vec(const b2pa_tensor* t, int dtype, int64_t n);
bool aligned16(const void* p);
bool pow2(int x);

struct Problem {
    int T, H, D, B, Hkv, P, N, max_pages, layout;
    bool fp8;
    long long q_st_tok, q_st_head, out_st_tok, out_st_head, bt_stride;
    long long k_st[3], v_st[3];  // page, head, slot (elements)
    const void *q, *k, *v;
    const int *bt, *seq, *cum_q, *cum_kv;
    int q_per_req;  // > 0: decode batch, request b owns query rows b * q_per_req .. (cum_q null)
    const int* kv_indptr;      // ragged page table: bt = the flat page ids, seq = derived on the device
    const int* last_page_len;
    const float* sinks;
    void* out;
};

int parse_pools(const b2pa_tensor* k, const b2pa_tensor* v, int32_t layout, Problem* pr);
int parse_problem(const b2pa_tensor* q, const b2pa_tensor* k_pool, const b2pa_tensor* v_pool,
                  const b2pa_tensor* block_tables, const b2pa_tensor* seq_lens, const b2pa_tensor* cum_q,
                  const b2pa_tensor* cum_kv, const b2pa_tensor* sinks, int32_t layout, const b2pa_tensor* out,
                  Problem* pr, int32_t q_per_req = 0, const b2pa_tensor* kv_indptr = nullptr,
                  const b2pa_tensor* last_page_len = nullptr);
// why the tensor-core paths cannot take this problem (nullptr if they can)
const char* tc_reject(const Problem& pr, const DevInfo& di);
// box: (64 columns, one kv head's query heads, rows_per_tile tokens)
int encode_q_map(CUtensorMap* m, const Problem& pr, int rows_per_tile);
int encode_pool_map(CUtensorMap* m, const Problem& pr, const void* base, const long long st[3]);

// (ops.cu) a scale tensor: the pool's shape without head_dim, fp32
int check_scales(const b2pa_tensor* s, const char* what, const b2pa_tensor* pool);

}  // namespace b2pa
