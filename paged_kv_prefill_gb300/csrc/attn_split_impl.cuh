// attn_split_impl.cuh -- the kernel and launch of attn_split.cuh, for the files that
// instantiate them.
#pragma once

#include "attn_split.cuh"

namespace b2pa {

namespace {

template <int D, bool FP8, int kTiles, int kSets>
struct SplitCfg {
    using Prefix = TreeCfg<D, FP8, kTiles>;
    static constexpr int kThreads = Prefix::kThreads;
    static constexpr int own_smem()
    {
        if constexpr (kSets == 0)
            return TreeCfg<D, FP8, 1>::kSmemBytes;
        else
            return FewCfg<D, FP8, kSets>::kSmemBytes;
    }
    static constexpr int kSmemBytes = Prefix::kSmemBytes > own_smem() ? Prefix::kSmemBytes : own_smem();
};

struct SplitRun : TreeRun {
    bool own;  // of the requests' own keys
};

// As tree_run, for two classes of work laid end to end, the prefixes' first: as many
// CTAs for either as its steps take of the time.  All numbers fit 32 bits (ops.cu); with
// 64-bit sums and divisions this took 4 us, a tenth of a batch's time.  `scan`: room for
// 68 numbers in shared memory that nothing else uses yet.
template <int kThreads, bool kWhole>
__device__ __forceinline__ SplitRun split_run(const TreeParams& p, int item_toks, int own_toks, int* scan)
{
    constexpr int kWarps = kThreads / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int groups = p.prefix.groups, n_req = groups + p.B;
    const int share = (n_req + kThreads - 1) / kThreads;
    const int b0 = min(n_req, tid * share), b1 = min(n_req, b0 + share);
    auto request = [&](int b) { return prefix_request(p, b, b < groups ? item_toks : own_toks); };
    auto work = [&](const TreeReq& r) { return r.items * p.Hkv * r.unit; };
    TreeReq r{};
    int mine = 0, shared = 0;  // steps; of them prefixes'
    for (int b = b0; b < b1; ++b) {
        r = request(b);
        if (!r.ok && blockIdx.x == 0)
            atomicOr(p.err, (unsigned)B2PA_DEV_BAD_REQUEST);
        mine += work(r);
        if (b < groups)
            shared += work(r);
    }
    int before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        before += lane >= o ? y : 0;
    }
    shared = __reduce_add_sync(0xffffffffu, shared);
    if (lane == 31) {
        scan[warp] = before;
        scan[32 + warp] = shared;
    }
    __syncthreads();
    int warps = lane < kWarps ? scan[lane] : 0;
    shared = __reduce_add_sync(0xffffffffu, lane < kWarps ? scan[32 + lane] : 0);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, warps, o);
        warps += lane >= o ? y : 0;
    }
    const int total = __shfl_sync(0xffffffffu, warps, 31), below = __shfl_sync(0xffffffffu, warps, max(warp - 1, 0));
    before += (warp > 0 ? below : 0) - mine;
    // CTAs by the time that the work takes, at least one for each class that has any
    const int grid = gridDim.x;
    const float a = p.prefix.step * (float)shared, b = (float)(total - shared);
    const int g = shared == 0       ? 0
                  : total == shared ? grid
                                    : min(grid - 1, max(1, __float2int_rn((float)grid * (a / (a + b)))));
    SplitRun run{};
    run.own = (int)blockIdx.x >= g;
    const int cta = (int)blockIdx.x - (run.own ? g : 0), steps = run.own ? total - shared : shared;
    // equal runs of two steps at least
    const int ctas = min(run.own ? grid - g : g, (steps + 1) / 2);
    const bool works = cta < ctas;
    const int each = works ? steps / ctas : 0, rest = steps - each * ctas;
    auto from = [&](int i) { return (run.own ? shared : 0) + each * i + (works ? rest * i / ctas : 0); };
    int start = works ? from(cta) : 0, end = works ? from(cta + 1) : 0;
    // by the threads whose requests the ends are in
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int x = k ? end : start;
        if (x < before || x >= before + mine)
            continue;
        int sum = before, q = b0;
        if (share > 1)
            r = request(q);
        for (; q + 1 < b1 && x >= sum + work(r); r = request(++q))
            sum += work(r);
        // (small units are not cut, where a cut costs more than a step)
        scan[64 + k] = kWhole || !run.own ? (int)tree_snap(x, sum, r, TreeCut{steps, ctas}, false) : x;
        if (k == 0) {
            scan[66] = sum;
            scan[67] = q;
        }
    }
    __syncthreads();
    if (works) {
        run.start = scan[64];
        run.end = end < total ? scan[65] : end;
        run.base = scan[66];
        run.first_b = scan[67];
    }
    fence_proxy_async_smem();  // later writes there come through the async proxy
    __syncthreads();
    return run;
}

template <int D, bool FP8, int kTiles, int kSets>
__global__ void __launch_bounds__(SplitCfg<D, FP8, kTiles, kSets>::kThreads, 1)
    prefix_split_kernel(const __grid_constant__ TreeParams p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    pdl_wait();
    const SplitRun run = split_run<SplitCfg<D, FP8, kTiles, kSets>::kThreads, kSets == 0>(
        p, kTiles * p.rows.tile_toks, p.rows.tile_toks, reinterpret_cast<int*>(smem));
    TreeCtx c;
    if (!run.own) {
        tree_setup<D, FP8, kTiles>(p, smem, c);
        tree_roles<D, FP8, kTiles, true>(p, c, run);
    } else if constexpr (kSets == 0) {
        tree_setup<D, FP8, 1>(p, smem, c);
        tree_roles<D, FP8, 1, true>(p, c, run);
    } else {
        few_setup<D, FP8, kSets>(p, smem, c);
        few_roles<D, FP8, kSets>(p, c, run);
    }
}

}  // namespace

template <int D, bool FP8, int kTiles, int kSets>
cudaError_t launch_split(const TreeParams& q, cudaStream_t stream)
{
    using C = SplitCfg<D, FP8, kTiles, kSets>;
    TreeParams p = q;
    // What steps take, found by timing.  Batch: 64 single tokens of 8 x 4 heads behind 16384
    // shared keys, bf16; groups: 100 of 8 x 8 heads in 8 groups, e4m3.
    //   step, batch: 2 / 2.5 / 3: 57 / 54 / 56 us;  groups: 3 / 3.75 / 4: 82.8 / 81.8 / 84.7, with 17
    //   requests each at least 115 / 107 / 110, with 16 at most (one query tile) 1.25 / 1.75 / 2 / 3: 76 / 64 / 66 / 73
    //   own_cost 1 / 2 / 3: batch 56 / 52 / 53, groups 99 / 86 / 89
    //   step, own keys by query tiles, batch: 0.75 / 1.5 / 2 / 3: 102 / 72 / 61 / 62
    if (kSets > 0) {
        p.prefix.own_cost = 2;
        p.prefix.step = kTiles == 2 ? (FP8 ? 3.75f : 2.5f) : FP8 ? 1.75f : 1.5f;
    } else {
        p.prefix.step = FP8 ? 1.5f : 2.f;
    }
    return launch_per_sm<prefix_split_kernel<D, FP8, kTiles, kSets>>(p, C::kThreads, C::kSmemBytes, stream);
}

}  // namespace b2pa
