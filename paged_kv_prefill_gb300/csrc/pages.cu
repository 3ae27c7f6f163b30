// pages.cu -- whole pages and single rows of the pools moved, and the ledger
// of which requests hold which pages.  Nothing is computed; what counts is the
// bytes that move and, for a decoding step's handful of rows, latency.
#include "pages.cuh"

#include <cooperative_groups.h>

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
// batch everything is read first.  Nothing but the places is shared between
// threads: a thread per node looks up where it comes from and where it goes.
// Latency: lengths, nodes, pages, rows, and the code itself.  256 requests of up to 24
// nodes, 2 KB each: 7.9 us; 8.5 with eight nodes at a time, 11.6 with 16; 8.4 with the
// pages looked up by every thread.
// ---------------------------------------------------------------------------
constexpr int kCompactThreads = 128;
constexpr int kCompactNodes = 32;  // whose places are looked up together

// Where a node comes from and goes to (from.x < 0: it stays).
struct Move {
    int from_page, from_slot, to_page, to_slot;
};

template <typename V>
__device__ __forceinline__ void compact_piece(const Plane& x, long long at, const Move* moves, int count)
{
    constexpr int kBatch = 4;
#pragma unroll 1
    for (int i0 = 0; i0 < count; i0 += kBatch) {
        V v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (i0 + k < count && moves[i0 + k].from_page >= 0) {
                const Move w = moves[i0 + k];
                v[k] = *reinterpret_cast<const V*>(x.base + (long long)w.from_page * x.st[0] + w.from_slot * x.st[2] + at);
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (i0 + k < count && moves[i0 + k].from_page >= 0) {
                const Move w = moves[i0 + k];
                *reinterpret_cast<V*>(x.base + (long long)w.to_page * x.st[0] + w.to_slot * x.st[2] + at) = v[k];
            }
        }
    }
}

__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const __grid_constant__ CompactParams p, int per)
{
    __shared__ Move moves[kCompactNodes];
    const int b = (int)(blockIdx.x / (unsigned)per), part = (int)(blockIdx.x - (unsigned)b * (unsigned)per);
    const int tid = threadIdx.x;
    pdl_wait();
    const int q0 = p.cum_q[b], n = p.cum_q[b + 1] - q0, kv = p.seq_lens[b], count = p.counts[b];
    const int* acc = p.accepted + (long long)b * p.acc_stride;
    bool bad = n < 0 || kv < n || count < 0 || count > n || count > p.width ||
               ((long long)kv + p.page_size - 1) / p.page_size > p.max_pages;
    int mine = 0;  // this thread's node of the first kCompactNodes
    if (!bad)
        for (int i = tid; i < count; i += kCompactThreads) {
            const int a = acc[i], before = i > 0 ? acc[i - 1] : -1;
            bad = bad || a <= before || a >= n;
            mine = i == tid ? a : mine;
        }
    bad = __syncthreads_or(bad);
    if (part == 0 && tid == 0) {
        p.new_lens[b] = bad ? kv : kv - n + count;
        if (bad)
            atomicOr(p.err, (unsigned)B2PA_DEV_BAD_REQUEST);
    }
    if (bad)
        return;
    int piece = part * kCompactThreads + tid;
    const bool on = piece < p.pieces;
    int plane = 0, per_row = p.plane[0].row / p.plane[0].vec;
    while (on && piece >= per_row * p.Hkv) {
        piece -= per_row * p.Hkv;
        ++plane;
        per_row = p.plane[plane].row / p.plane[plane].vec;
    }
    const Plane& x = p.plane[plane];
    const int head = piece / per_row;
    const long long at = head * x.st[1] + (long long)(piece - head * per_row) * x.vec;
    const int* pages = p.block_tables + (long long)b * p.bt_stride;
    const int ctx = kv - n;
    for (int i0 = 0; i0 < count; i0 += kCompactNodes) {
        const int some = min(kCompactNodes, count - i0);
        if (tid < some) {
            const int i = i0 + tid, a = i0 == 0 ? mine : acc[i];
            Move w{-1, 0, 0, 0};
            if (a != i) {
                const int from = (ctx + a) / p.page_size, to = (ctx + i) / p.page_size;
                w = Move{pages[from], ctx + a - from * p.page_size, pages[to], ctx + i - to * p.page_size};
                if (w.from_page < 0 || w.from_page >= p.num_pages || w.to_page < 0 || w.to_page >= p.num_pages) {
                    atomicOr(p.err, (unsigned)B2PA_DEV_BAD_PAGE);
                    w.from_page = -1;
                }
            }
            moves[tid] = w;
        }
        __syncthreads();
        if (on)
            switch (x.vec) {
            case 16: compact_piece<uint4>(x, at, moves, some); break;
            case 8: compact_piece<uint2>(x, at, moves, some); break;
            case 4: compact_piece<uint32_t>(x, at, moves, some); break;
            case 2: compact_piece<uint16_t>(x, at, moves, some); break;
            default: compact_piece<uint8_t>(x, at, moves, some);
            }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// The ledger.  A page is free if its count is 0.
// ---------------------------------------------------------------------------
__device__ __forceinline__ int pages_of(int tokens, int page_size) { return (int)(((long long)tokens + page_size - 1) / page_size); }

// A page loses a holder.  (Only such calls may be under way for the page, and a count
// that would fall below 0 is put back, so that their order does not show.)
__device__ __forceinline__ void give_back(const LedgerParams& p, int page)
{
    if (page < 0 || page >= p.N) {
        atomicOr(p.err, (unsigned)B2PA_DEV_BAD_PAGE);
    } else if (atomicSub(p.refs + page, 1) <= 0) {
        atomicAdd(p.refs + page, 1);
        atomicOr(p.err, (unsigned)B2PA_DEV_BAD_PAGE);
    }
}

constexpr int kFreeThreads = 128;

// A block per row.
__global__ void __launch_bounds__(kFreeThreads) free_pages_kernel(const __grid_constant__ LedgerParams p)
{
    __shared__ int held;
    pdl_wait();
    const int r = p.rows[blockIdx.x], tid = threadIdx.x;
    const bool in = r >= 0 && r < p.R;
    const int* row = p.tables + (long long)r * p.stride;
    int page = in && tid < p.max_pages ? row[tid] : 0;  // (while the length is on its way)
    if (tid == 0) {
        int len = in ? p.seq[r] : -1;
        if (len < 0 || pages_of(len, p.page_size) > p.max_pages) {
            atomicOr(p.err, (unsigned)B2PA_DEV_BAD_REQUEST);
            len = 0;
        } else if (len > 0) {
            len = atomicExch(p.seq + r, 0);  // (a row named twice is freed once)
        }
        held = pages_of(len, p.page_size);
    }
    __syncthreads();
    for (int c = tid; c < held; c += kFreeThreads) {
        page = c == tid ? page : row[c];
        give_back(p, page);
    }
}

// Fork and grow: each request wants some pages, and gets the lowest free ones,
// in the order of the requests.  One cluster: what the requests want, summed up (by
// every CTA); the free pages counted, each CTA those of its part of the pool; then
// whoever finds the k-th free page looks up whose it is.  A request of which some
// page would be missing gets none; pages that rows give back are free from the next
// call on.  Bound by latency: about ten dependent accesses to
// memory and shared memory.  16 samples each of 16 prompts, free, fork, grow and copy:
// 27.3 us (of which the copy takes 9) with eight CTAs, 45.9 with one, 30.8 with four; a thread
// that looks up all of its 16 free pages one after the other: 42.
constexpr int kTakeThreads = 1024;
constexpr int kTakeWarps = kTakeThreads / 32;
static_assert(kTakeWarps == 32, "block_scan: a sum per lane");
constexpr int kTakeRun = 16;  // pages that a thread looks at, one behind the other
constexpr int kTakeCtas = 8;  // of a cluster at most
constexpr int kTakeList = 2048;  // pages that are given away together

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

// Which of the pages i .. i + kTakeRun - 1, below end, are free.
__device__ __forceinline__ unsigned free_bits(const int* refs, int i, int end, bool aligned)
{
    unsigned bits = 0;
    if (aligned && i + kTakeRun <= end) {
        int4 x[kTakeRun / 4];
#pragma unroll
        for (int k = 0; k < kTakeRun / 4; ++k)
            x[k] = reinterpret_cast<const int4*>(refs + i)[k];
#pragma unroll
        for (int k = 0; k < kTakeRun / 4; ++k)
            bits |= (unsigned)(x[k].x == 0) << 4 * k | (unsigned)(x[k].y == 0) << (4 * k + 1) |
                    (unsigned)(x[k].z == 0) << (4 * k + 2) | (unsigned)(x[k].w == 0) << (4 * k + 3);
    } else {
#pragma unroll
        for (int k = 0; k < kTakeRun; ++k)
            if (i + k < end)
                bits |= (unsigned)(refs[i + k] == 0) << k;
    }
    return bits;
}

template <bool kFork>
__global__ void __launch_bounds__(kTakeThreads) take_pages_kernel(const __grid_constant__ LedgerParams p)
{
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ int words[];  // [n + 1] each:
    int* off = words;               // pages that the requests before want
    int* base = off + p.n + 1;      // twice a request's first new column, plus 1 if it wants any; -1: malformed
    int* rows = base + p.n + 1;     // the call's rows
    int* parents = rows + p.n + 1;  // fork: and their parents
    __shared__ int list[kTakeList];
    __shared__ int sums[32];
    __shared__ int counts[kTakeCtas];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    pdl_wait();
    for (int i = tid; i < p.n; i += kTakeThreads) {
        rows[i] = p.rows[i];
        if (kFork)
            parents[i] = p.parents[i];
    }
    // the free pages of this CTA's part, the first of it kept
    constexpr int kTile = kTakeThreads * kTakeRun;
    const int part = ((p.N + ctas - 1) / ctas + kTakeRun - 1) / kTakeRun * kTakeRun;
    const int first = (int)min((long long)p.N, (long long)rank * part), end = min(p.N, first + part);
    const bool aligned = (reinterpret_cast<uintptr_t>(p.refs) & 15u) == 0;
    const unsigned kept = free_bits(p.refs, first + tid * kTakeRun, end, aligned);
    int mine = __popc(kept), before;
    for (int i = first + kTile + tid * kTakeRun; i < end; i += kTile)
        mine += __popc(free_bits(p.refs, i, end, aligned));
    // what each request wants
    for (int i = tid; i < p.n; i += kTakeThreads) {
        const int r = rows[i];
        int col = -1, want = 0;
        if (r >= 0 && r < p.R) {
            const int have = p.seq[r];
            if (kFork) {
                const int from = parents[i];
                const int len = from >= 0 && from < p.R ? p.seq[from] : -1;
                if (have == 0 && len >= 0 && pages_of(len, p.page_size) <= p.max_pages) {
                    col = len / p.page_size;
                    want = len % p.page_size != 0;
                }
            } else {
                const int to = p.to[i];
                if (have >= 0 && to >= 0 && pages_of(max(have, to), p.page_size) <= p.max_pages) {
                    col = pages_of(have, p.page_size);
                    want = max(pages_of(to, p.page_size) - col, 0);
                }
            }
        }
        base[i] = col < 0 ? -1 : 2 * col + (want > 0);
        off[i] = want;
    }
    const int found = block_scan(mine, sums, &before);
    if (ctas > 1)
        cluster.sync();  // (from here on CTAs write one another's shared memory)
    if (tid < ctas)
        *cluster.map_shared_rank(&counts[rank], tid) = found;
    // a row is named once, and nobody forks a row that is written (a warp per request)
    for (int i = rank * kTakeWarps + warp; i < p.n; i += ctas * kTakeWarps) {
        const int r = rows[i];
        bool clash = false;
#pragma unroll 4
        for (int j = lane; j < p.n; j += 32)
            clash |= (j < i && rows[j] == r) || (kFork && parents[j] == r);
        clash = __any_sync(0xffffffffu, clash);
        if (clash || base[i] < 0) {
            if (lane < ctas) {
                *cluster.map_shared_rank(&base[i], lane) = -1;
                *cluster.map_shared_rank(&off[i], lane) = 0;
            }
            if (lane == 0)
                atomicOr(p.err, (unsigned)B2PA_DEV_BAD_REQUEST);
        }
    }
    if (ctas > 1)
        cluster.sync();
    else
        __syncthreads();
    int total = 0, avail = 0, lower = 0;
    for (int i = 0; i < ctas; ++i) {
        lower = i == rank ? avail : lower;
        avail += counts[i];
    }
    for (int i0 = 0; i0 < p.n; i0 += kTakeThreads) {
        const int i = i0 + tid, want = i < p.n ? off[i] : 0;
        int sum;
        const int all = block_scan(want, sums, &sum);
        if (i < p.n)
            off[i] = add(total, sum);
        total = add(total, all);
    }
    if (tid == 0)
        off[p.n] = total;
    __syncthreads();
    // whose the free pages are
    const int give = min(total, avail);
    for (int i0 = first, k0 = lower; i0 < end && k0 < give; i0 += kTile) {
        const int i = i0 + tid * kTakeRun;
        unsigned bits = kept;
        int all = 0;
        if (part > kTile) {
            bits = i0 == first ? kept : i < end ? free_bits(p.refs, i, end, aligned) : 0u;
            all = block_scan(__popc(bits), sums, &before);
        }
        // the k0-th free page and those behind it, in lists (they lie close together, and
        // looking up whose a page is takes a while: one thread per page)
        const int some = min(part > kTile ? all : found, give - k0);
        for (int l0 = 0; l0 < some; l0 += kTakeList) {
            int k = before - l0;
            for (unsigned x = bits; x != 0 && k < kTakeList; x &= x - 1, ++k)
                if (k >= 0)
                    list[k] = i + __ffs(x) - 1;
            __syncthreads();
            for (int l = tid; l < min(kTakeList, some - l0); l += kTakeThreads) {
                const int page = list[l], nth = k0 + l0 + l;
                int lo = 0, hi = p.n - 1;  // the last request with off <= nth
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (off[mid] <= nth)
                        lo = mid;
                    else
                        hi = mid - 1;
                }
                if (off[lo + 1] > avail)
                    continue;  // not all of this request's
                const int col = (base[lo] >> 1) + (nth - off[lo]);
                p.tables[(long long)rows[lo] * p.stride + col] = page;
                p.refs[page] = 1;
                if (kFork)
                    p.dst[lo] = page;
            }
            __syncthreads();
        }
        k0 += all;
    }
    if (part > kTile && ctas > 1)
        cluster.sync();  // (counts have been read: what follows writes them)
    else if (part > kTile)
        __syncthreads();
    // what is left to do for each request, a warp each
    for (int i = rank * kTakeWarps + warp; i < p.n; i += ctas * kTakeWarps) {
        const bool bad = base[i] < 0, wants = !bad && (base[i] & 1), none = wants && off[i + 1] > avail;
        if (none && lane == 0)
            atomicOr(p.err, (unsigned)B2PA_DEV_NO_PAGES);
        if (kFork) {
            const bool rest = wants && !none;
            const int from = parents[i], r = rows[i], whole = base[i] >> 1;
            const int* in = p.tables + (long long)from * p.stride;
            if (lane == 0) {
                const int page = rest ? in[whole] : -1;
                p.src[i] = page;
                if (!rest)
                    p.dst[i] = -1;
                else if (page < 0 || page >= p.N)
                    atomicOr(p.err, (unsigned)B2PA_DEV_BAD_PAGE);
            }
            if (bad || none)
                continue;
            if (lane == 0)
                p.seq[r] = p.seq[from];
            int* out = p.tables + (long long)r * p.stride;
            constexpr int kBatch = 8;
            for (int c0 = lane; c0 < whole; c0 += 32 * kBatch) {
                int page[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
                    page[k] = c0 + 32 * k < whole ? in[c0 + 32 * k] : -1;
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    if (c0 + 32 * k >= whole)
                        break;
                    out[c0 + 32 * k] = page[k];
                    if (page[k] < 0 || page[k] >= p.N)
                        atomicOr(p.err, (unsigned)B2PA_DEV_BAD_PAGE);
                    else
                        atomicAdd(p.refs + page[k], 1);
                }
            }
        } else if (!bad && !none) {
            const int r = rows[i], to = p.to[i];
            if (lane == 0)
                p.seq[r] = to;
            // pages that a shorter row gives back
            for (int c = pages_of(to, p.page_size) + lane; c < base[i] >> 1; c += 32)
                give_back(p, p.tables[(long long)r * p.stride + c]);
        }
    }
}

// `cluster` CTAs to a cluster
template <typename Kern, typename... Args>
cudaError_t launch(Kern kern, unsigned grid, unsigned threads, unsigned cluster, size_t smem, cudaStream_t stream,
                   const Args&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {cluster, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <bool kFork>
cudaError_t launch_take(const LedgerParams& p, cudaStream_t stream)
{
    const size_t smem = 4 * ((size_t)p.n + 1) * sizeof(int);
    if (smem > 32 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(take_pages_kernel<kFork>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   4 * (kLedgerMax + 1) * (int)sizeof(int));
        if (e != cudaSuccess)
            return e;
    }
    // one CTA for a few requests and a pool that it looks through at once (4 beams of
    // 2000 pages, the four calls: 14.6 us; 16.5 with a cluster of eight)
    const unsigned ctas = p.n <= kTakeWarps && p.N <= kTakeThreads * kTakeRun ? 1 : kTakeCtas;
    return launch(take_pages_kernel<kFork>, ctas, kTakeThreads, ctas, smem, stream, p);
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
    return launch(copy_pages_kernel, (unsigned)(per * p.n), kCopyThreads, 1, 0, stream, p);
}

cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream)
{
    const long long per = (p.pieces + kCompactThreads - 1) / kCompactThreads;
    if (per * p.B > 0x7FFFFFFFLL)
        return cudaErrorInvalidConfiguration;
    return launch(compact_kernel, (unsigned)(per * p.B), kCompactThreads, 1, 0, stream, p, (int)per);
}

cudaError_t launch_free_pages(const LedgerParams& p, cudaStream_t stream)
{
    return launch(free_pages_kernel, (unsigned)p.n, kFreeThreads, 1, 0, stream, p);
}

cudaError_t launch_take_pages(const LedgerParams& p, bool fork, cudaStream_t stream)
{
    return fork ? launch_take<true>(p, stream) : launch_take<false>(p, stream);
}

}  // namespace b2pa
