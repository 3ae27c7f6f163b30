// pages.cu -- whole pages and single rows of the pools moved, and the ledger
// of which requests hold which pages.  Nothing is computed; what counts is the
// bytes that move and, for a decoding step's handful of rows, latency.
#include "pages.cuh"

#include "../../include/b2pa.h"
#include "ptx.cuh"

namespace b2pa {

namespace {

// ---------------------------------------------------------------------------
// Pages src[i] -> dst[i].  A block moves kCopyPieces pieces per thread of one
// plane of one page, all loads before the stores.
// ---------------------------------------------------------------------------
constexpr int kCopyThreads = 256;
constexpr int kCopyPieces = 4;

template <typename V>
__device__ __forceinline__ void copy_pieces(const CopyPagesParams& p, int plane, const uint8_t* from, uint8_t* to, int block)
{
    const long long pieces = p.row[plane] / (long long)sizeof(V);  // of a row
    const long long all = pieces * p.inner[plane] * p.outer[plane];
    V x[kCopyPieces];
    long long at[kCopyPieces];
#pragma unroll
    for (int k = 0; k < kCopyPieces; ++k) {
        const long long i = ((long long)block * kCopyPieces + k) * kCopyThreads + threadIdx.x;
        at[k] = -1;
        if (i < all) {
            at[k] = i * (long long)sizeof(V);
            if (p.inner[plane] * p.outer[plane] > 1) {  // (a page fits 32 bits many times)
                const unsigned row = (unsigned)i / (unsigned)pieces, in = (unsigned)i - row * (unsigned)pieces;
                const unsigned o = row / (unsigned)p.inner[plane], r = row - o * (unsigned)p.inner[plane];
                at[k] = o * p.outer_st[plane] + r * p.inner_st[plane] + (long long)in * (long long)sizeof(V);
            }
            x[k] = *reinterpret_cast<const V*>(from + at[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < kCopyPieces; ++k)
        if (at[k] >= 0)
            *reinterpret_cast<V*>(to + at[k]) = x[k];
}

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyPagesParams p)
{
    int per = 0;
    for (int k = 0; k < p.planes; ++k)
        per += p.blocks[k];
    const int pair = (int)(blockIdx.x / (unsigned)per);
    int block = (int)(blockIdx.x - (unsigned)pair * (unsigned)per), plane = 0;
    while (block >= p.blocks[plane])
        block -= p.blocks[plane++];
    pdl_wait();
    const int src = p.src[pair], dst = p.dst[pair];
    if (src == -1 && dst == -1)
        return;  // nothing to copy
    if (src < 0 || src >= p.num_pages || dst < 0 || dst >= p.num_pages) {
        if (block == 0 && plane == 0 && threadIdx.x == 0)
            atomicOr(p.err, (unsigned)B2PA_DEV_BAD_PAGE);
        return;
    }
    const Plane& x = p.plane[plane];
    const uint8_t* from = x.base + (long long)src * x.st[0];
    uint8_t* to = x.base + (long long)dst * x.st[0];
    switch (x.vec) {
    case 16: copy_pieces<uint4>(p, plane, from, to, block); break;
    case 8: copy_pieces<uint2>(p, plane, from, to, block); break;
    case 4: copy_pieces<uint32_t>(p, plane, from, to, block); break;
    case 2: copy_pieces<uint16_t>(p, plane, from, to, block); break;
    default: copy_pieces<uint8_t>(p, plane, from, to, block);
    }
}

// ---------------------------------------------------------------------------
// Rows of the accepted nodes to the first places behind the context.  A thread
// owns one piece of a token's rows and moves it for node after node, kBatch
// nodes at a time: node i goes to place i from place a_i >= i, and the a_i
// rise, so that what a batch overwrites no later node comes from, and within a
// batch everything is read first.  Nothing is shared between threads.
// ---------------------------------------------------------------------------
constexpr int kCompactThreads = 128;

template <typename V>
__device__ __forceinline__ void compact_piece(const CompactParams& p, const Plane& x, long long at, const int* pages,
                                              const int* acc, int ctx, int count)
{
    constexpr int kBatch = 8;
    auto place = [&](int token, bool* ok) -> uint8_t* {
        const int col = token / p.page_size, slot = token - col * p.page_size;
        const int page = pages[col];
        *ok = page >= 0 && page < p.num_pages;
        return x.base + (long long)page * x.st[0] + slot * x.st[2] + at;
    };
    for (int i0 = 0; i0 < count; i0 += kBatch) {
        V v[kBatch];
        uint8_t* to[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            to[k] = nullptr;
            if (i0 + k < count) {
                const int a = acc[i0 + k];
                if (a != i0 + k) {
                    bool ok_from, ok_to;
                    const uint8_t* from = place(ctx + a, &ok_from);
                    uint8_t* dst = place(ctx + i0 + k, &ok_to);
                    if (ok_from && ok_to) {
                        to[k] = dst;
                        v[k] = *reinterpret_cast<const V*>(from);
                    } else {
                        atomicOr(p.err, (unsigned)B2PA_DEV_BAD_PAGE);
                    }
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (to[k] != nullptr)
                *reinterpret_cast<V*>(to[k]) = v[k];
    }
}

__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const __grid_constant__ CompactParams p, int per)
{
    const int b = (int)(blockIdx.x / (unsigned)per), part = (int)(blockIdx.x - (unsigned)b * (unsigned)per);
    pdl_wait();
    const int q0 = p.cum_q[b], n = p.cum_q[b + 1] - q0, kv = p.seq_lens[b], count = p.counts[b];
    const int* acc = p.accepted + (long long)b * p.acc_stride;
    bool bad = n < 0 || kv < n || count < 0 || count > n || count > p.width ||
               ((long long)kv + p.page_size - 1) / p.page_size > p.max_pages;
    if (!bad)
        for (int i = threadIdx.x; i < count; i += kCompactThreads) {
            const int a = acc[i], before = i > 0 ? acc[i - 1] : -1;
            bad = bad || a <= before || a >= n;
        }
    bad = __syncthreads_or(bad);
    if (part == 0 && threadIdx.x == 0) {
        p.new_lens[b] = bad ? kv : kv - n + count;
        if (bad)
            atomicOr(p.err, (unsigned)B2PA_DEV_BAD_REQUEST);
    }
    int piece = part * kCompactThreads + (int)threadIdx.x;
    if (bad || piece >= p.pieces)
        return;
    int plane = 0, per_row = p.plane[0].row / p.plane[0].vec;
    while (piece >= per_row * p.Hkv) {
        piece -= per_row * p.Hkv;
        ++plane;
        per_row = p.plane[plane].row / p.plane[plane].vec;
    }
    const Plane& x = p.plane[plane];
    const int head = piece / per_row;
    const long long at = head * x.st[1] + (long long)(piece - head * per_row) * x.vec;
    const int* pages = p.block_tables + (long long)b * p.bt_stride;
    switch (x.vec) {
    case 16: compact_piece<uint4>(p, x, at, pages, acc, kv - n, count); break;
    case 8: compact_piece<uint2>(p, x, at, pages, acc, kv - n, count); break;
    case 4: compact_piece<uint32_t>(p, x, at, pages, acc, kv - n, count); break;
    case 2: compact_piece<uint16_t>(p, x, at, pages, acc, kv - n, count); break;
    default: compact_piece<uint8_t>(p, x, at, pages, acc, kv - n, count);
    }
}

// ---------------------------------------------------------------------------
// The ledger.  A page is free if its count is 0.
// ---------------------------------------------------------------------------
__device__ __forceinline__ int pages_of(int tokens, int page_size) { return (int)(((long long)tokens + page_size - 1) / page_size); }

constexpr int kFreeThreads = 128;

// A block per row.  (Counts only fall here, and a count that would fall below 0
// is put back, so that the order of the blocks does not show.)
__global__ void __launch_bounds__(kFreeThreads) free_pages_kernel(const __grid_constant__ LedgerParams p)
{
    __shared__ int held;
    pdl_wait();
    const int r = p.rows[blockIdx.x];
    if (threadIdx.x == 0) {
        int len = r >= 0 && r < p.R ? p.seq[r] : -1;
        if (len < 0 || pages_of(len, p.page_size) > p.max_pages) {
            atomicOr(p.err, (unsigned)B2PA_DEV_BAD_REQUEST);
            len = 0;
        } else if (len > 0) {
            len = atomicExch(p.seq + r, 0);  // (a row named twice is freed once)
        }
        held = pages_of(len, p.page_size);
    }
    __syncthreads();
    const int* row = p.tables + (long long)r * p.stride;
    for (int c = threadIdx.x; c < held; c += kFreeThreads) {
        const int page = row[c];
        if (page < 0 || page >= p.N) {
            atomicOr(p.err, (unsigned)B2PA_DEV_BAD_PAGE);
        } else if (atomicSub(p.refs + page, 1) <= 0) {
            atomicAdd(p.refs + page, 1);
            atomicOr(p.err, (unsigned)B2PA_DEV_BAD_PAGE);
        }
    }
}

// Fork and grow: each request wants some pages, and gets the lowest free ones,
// in the order of the requests.  One block: what the requests want, summed up;
// the free pages counted; then whoever finds the k-th free page looks up whose
// it is.  A request of which some page would be missing gets none.
constexpr int kTakeThreads = 1024;

// Sums end at kLots, which is more than any number of pages (ops_pages.cu).
constexpr int kLots = 0x3FFFFFFF;
__device__ __forceinline__ int add(int a, int b) { return min(a + b, kLots); }

// Sum over the block of x <= kLots; `before` gets that of the threads before this one.
__device__ __forceinline__ int block_scan(int x, int* warps /* [32] in shared memory */, int* before)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, o);
        y = add(y, lane >= o ? z : 0);
    }
    __syncthreads();  // (the last call's sums have been read)
    if (lane == 31)
        warps[warp] = y;
    __syncthreads();
    if (warp == 0) {
        int w = warps[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, w, o);
            w = add(w, lane >= o ? z : 0);
        }
        warps[lane] = w;
    }
    const int in_warp = __shfl_up_sync(0xffffffffu, y, 1);
    __syncthreads();
    *before = add(lane > 0 ? in_warp : 0, warp > 0 ? warps[warp - 1] : 0);
    return warps[31];
}

template <bool kFork>
__global__ void __launch_bounds__(kTakeThreads) take_pages_kernel(const __grid_constant__ LedgerParams p)
{
    __shared__ int off[kLedgerMax + 1];  // pages that the requests before want
    __shared__ int base[kLedgerMax];     // twice a request's first new column, plus 1 if it wants any; -1: malformed
    __shared__ int sums[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    // what each request wants
    for (int i = tid; i < p.n; i += kTakeThreads) {
        const int r = p.rows[i];
        int first = -1, want = 0;
        if (r >= 0 && r < p.R) {
            if (kFork) {
                const int from = p.parents[i];
                const int len = from >= 0 && from < p.R && p.seq[r] == 0 ? p.seq[from] : -1;
                if (len >= 0 && pages_of(len, p.page_size) <= p.max_pages) {
                    first = len / p.page_size;
                    want = len % p.page_size != 0;
                }
            } else {
                const int len = p.seq[r], to = p.to[i];
                if (len >= 0 && to >= len && pages_of(to, p.page_size) <= p.max_pages) {
                    first = pages_of(len, p.page_size);
                    want = pages_of(to, p.page_size) - first;
                }
            }
        }
        base[i] = first < 0 ? -1 : 2 * first + (want > 0);
        off[i] = want;
    }
    __syncthreads();
    // a row is named once, and nobody forks a row that is written (a warp per request)
    for (int i = warp; i < p.n; i += kTakeThreads / 32) {
        const int r = p.rows[i];
        bool clash = false;
        for (int j = lane; j < p.n; j += 32)
            clash = clash || (j < i && p.rows[j] == r) || (kFork && p.parents[j] == r);
        clash = __any_sync(0xffffffffu, clash);
        if (lane == 0 && (clash || base[i] < 0)) {
            base[i] = -1;
            off[i] = 0;
            atomicOr(p.err, (unsigned)B2PA_DEV_BAD_REQUEST);
        }
    }
    __syncthreads();
    int total = 0;
    for (int i0 = 0; i0 < p.n; i0 += kTakeThreads) {
        const int i = i0 + tid, want = i < p.n ? off[i] : 0;
        int before;
        const int all = block_scan(want, sums, &before);
        if (i < p.n)
            off[i] = add(total, before);
        total = add(total, all);
    }
    if (tid == 0)
        off[p.n] = total;
    // how many are free
    int mine = 0, before;
    for (int i = tid; i < p.N; i += kTakeThreads)
        mine += p.refs[i] == 0;
    const int avail = block_scan(mine, sums, &before);  // (its barriers: off is complete)
    // whose the free pages are
    const int give = min(total, avail);
    for (int i0 = 0, found = 0; i0 < p.N && found < give; i0 += kTakeThreads) {
        const int page = i0 + tid;
        const bool free = page < p.N && p.refs[page] == 0;
        const int all = block_scan(free, sums, &before);
        const int k = found + before;
        found += all;
        if (!free || k >= give)
            continue;
        int lo = 0, hi = p.n - 1;  // the last request with off <= k
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (off[mid] <= k)
                lo = mid;
            else
                hi = mid - 1;
        }
        if (off[lo + 1] > avail)
            continue;  // not all of this request's
        const int col = (base[lo] >> 1) + (k - off[lo]);
        p.tables[(long long)p.rows[lo] * p.stride + col] = page;
        p.refs[page] = 1;
        if (kFork)
            p.dst[lo] = page;
    }
    __syncthreads();
    // what is left to do for each request, a warp each
    for (int i = warp; i < p.n; i += kTakeThreads / 32) {
        const bool bad = base[i] < 0, wants = !bad && (base[i] & 1), none = wants && off[i + 1] > avail;
        if (none && lane == 0)
            atomicOr(p.err, (unsigned)B2PA_DEV_NO_PAGES);
        if (kFork) {
            const bool part = wants && !none;
            const int from = p.parents[i], r = p.rows[i], whole = base[i] >> 1;
            const int* in = p.tables + (long long)from * p.stride;
            if (lane == 0) {
                p.src[i] = part ? in[whole] : -1;
                if (!part)
                    p.dst[i] = -1;
            }
            if (bad || none)
                continue;
            int* out = p.tables + (long long)r * p.stride;
            for (int c = lane; c < whole; c += 32) {
                const int page = in[c];
                out[c] = page;
                if (page < 0 || page >= p.N)
                    atomicOr(p.err, (unsigned)B2PA_DEV_BAD_PAGE);
                else
                    atomicAdd(p.refs + page, 1);
            }
            if (lane == 0)
                p.seq[r] = p.seq[from];
        } else if (!bad && !none && lane == 0) {
            p.seq[p.rows[i]] = p.to[i];
        }
    }
}

template <typename Kern, typename... Args>
cudaError_t launch(Kern kern, unsigned grid, unsigned threads, cudaStream_t stream, const Args&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace

cudaError_t launch_copy_pages(const CopyPagesParams& q, cudaStream_t stream)
{
    CopyPagesParams p = q;
    long long per = 0;
    for (int k = 0; k < p.planes; ++k) {
        const long long pieces = p.row[k] / p.plane[k].vec * p.inner[k] * p.outer[k];
        const long long blocks = (pieces + kCopyThreads * kCopyPieces - 1) / (kCopyThreads * kCopyPieces);
        if (blocks > 0x7FFFFFFF)
            return cudaErrorInvalidConfiguration;
        p.blocks[k] = (int)blocks;
        per += blocks;
    }
    if (per * p.n > 0x7FFFFFFFLL)
        return cudaErrorInvalidConfiguration;
    return launch(copy_pages_kernel, (unsigned)(per * p.n), kCopyThreads, stream, p);
}

cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream)
{
    const long long per = (p.pieces + kCompactThreads - 1) / kCompactThreads;
    if (per * p.B > 0x7FFFFFFFLL)
        return cudaErrorInvalidConfiguration;
    return launch(compact_kernel, (unsigned)(per * p.B), kCompactThreads, stream, p, (int)per);
}

cudaError_t launch_free_pages(const LedgerParams& p, cudaStream_t stream)
{
    return launch(free_pages_kernel, (unsigned)p.n, kFreeThreads, stream, p);
}

cudaError_t launch_take_pages(const LedgerParams& p, bool fork, cudaStream_t stream)
{
    return fork ? launch(take_pages_kernel<true>, 1, kTakeThreads, stream, p)
                : launch(take_pages_kernel<false>, 1, kTakeThreads, stream, p);
}

}  // namespace b2pa
