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
    static constexpr int kOne = TreeCfg<D, FP8, 1>::kSmemBytes;
    static constexpr int own_smem()
    {
        if constexpr (kSets == 0)
            return kOne;
        else
            return FewCfg<D, FP8, kSets>::kSmemBytes;
    }
    static constexpr int kOthers = own_smem() > kOne ? own_smem() : kOne;
    static constexpr int kSmemBytes = Prefix::kSmemBytes > kOthers ? Prefix::kSmemBytes : kOthers;
};

// What a CTA works on: prefixes with two query tiles, prefixes with one, the requests' own
// keys.  kTiles 2: over an e4m3 cache prefixes of no more rows than one query tile are the
// second kind, with both softmax groups on it (the groups below: 77 us, 82 without); over a
// bf16 cache they are the first (their share is smaller: 101 us, 105 apart).
enum SplitKind { kTwoTiles, kOneTile, kOwnKeys };

struct SplitRun : TreeRun {
    int kind;
};

// As tree_run, for each kind of work by itself: as many CTAs as its steps take of the
// time.  All numbers fit 32 bits (ops.cu); with 64-bit sums and divisions this took 4 us, a
// tenth of a batch's time.  `scan`: room for 52 numbers in shared memory that nothing
// else uses yet.
template <int kThreads, int kTiles, bool FP8, bool kWhole>
__device__ __forceinline__ SplitRun split_run(const TreeParams& p, int* scan)
{
    constexpr int kWarps = kThreads / 32;
    constexpr bool kTwo = kTiles == 2, kOne = kTiles == 1 || FP8;  // the kinds of prefixes that there are
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, tile = p.rows.tile_toks;
    const int groups = p.prefix.groups, n_req = groups + p.B;
    const int share = (n_req + kThreads - 1) / kThreads;
    const int b0 = min(n_req, tid * share), b1 = min(n_req, b0 + share);
    int kind = 0;  // of the last request
    auto request = [&](int b) {
        TreeReq r = prefix_request(p, b, tile);
        kind = b >= groups ? kOwnKeys : kTiles == 2 && (!FP8 || r.n > tile) ? kTwoTiles : kOneTile;
        if (kind == kTwoTiles)
            r.items = (r.items + 1) / 2;
        return r;
    };
    auto work = [&](const TreeReq& r) { return r.items * p.Hkv * r.unit; };
    TreeReq r{};
    int mine[3] = {0, 0, 0}, before[3], total[3] = {0, 0, 0};  // steps: this thread's, those before, all
    for (int b = b0; b < b1; ++b) {
        r = request(b);
        if (!r.ok && blockIdx.x == 0)
            atomicOr(p.err, (unsigned)B2PA_DEV_BAD_REQUEST);
        const int w = work(r);
        mine[0] += kTwo && kind == kTwoTiles ? w : 0;
        mine[1] += kOne && kind == kOneTile ? w : 0;
        mine[2] += kind == kOwnKeys ? w : 0;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        before[k] = mine[k];
        if ((k == 0 && !kTwo) || (k == 1 && !kOne))
            continue;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, before[k], o);
            before[k] += lane >= o ? y : 0;
        }
        if (lane == 31)
            scan[16 * k + warp] = before[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        if ((k == 0 && !kTwo) || (k == 1 && !kOne))
            continue;
        const int x = lane < kWarps ? scan[16 * k + lane] : 0;
        total[k] = __reduce_add_sync(0xffffffffu, x);
        before[k] += __reduce_add_sync(0xffffffffu, lane < warp ? x : 0) - mine[k];
    }
    // CTAs by the time that the work takes, at least one for each kind that has any
    const int grid = gridDim.x;
    const float a0 = p.prefix.step[0] * (float)total[0], a1 = p.prefix.step[1] * (float)total[1];
    const float per = (float)grid / (a0 + a1 + (float)total[2]);  // (not a number: there is nothing to do)
    const int some1 = total[1] > 0, some2 = total[2] > 0;
    const int n0 = total[0] > 0 ? min(grid - some1 - some2, max(1, __float2int_rn(per * a0))) : 0;
    const int n1 = !some1 ? 0 : !some2 ? grid - n0 : min(grid - n0 - 1, max(1, __float2int_rn(per * a1)));
    const int cta_id = blockIdx.x;
    SplitRun run{};
    run.kind = kTwo && cta_id < n0 ? kTwoTiles : kOne && cta_id < n0 + n1 ? kOneTile : kOwnKeys;
    auto of_kind = [&](int x0, int x1, int x2) {
        return kTwo && run.kind == kTwoTiles ? x0 : kOne && run.kind == kOneTile ? x1 : x2;
    };
    const int cta = cta_id - of_kind(0, n0, n0 + n1), steps = of_kind(total[0], total[1], total[2]);
    // equal runs of two steps at least
    const int ctas = min(of_kind(n0, n1, grid - n0 - n1), (steps + 1) / 2);
    const bool works = cta < ctas;
    const int each = works ? steps / ctas : 0, rest = steps - each * ctas;
    auto from = [&](int i) { return each * i + (works ? rest * i / ctas : 0); };
    const int start = works ? from(cta) : 0, end = works ? from(cta + 1) : 0;
    const int first = of_kind(before[0], before[1], before[2]), here = of_kind(mine[0], mine[1], mine[2]);
    // by the threads whose requests the ends are in
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int x = k ? end : start;
        if (x < first || x >= first + here)
            continue;
        int sum = first, q = b0;
        if (share > 1)
            r = request(q);
        for (int w; q + 1 < b1 && x >= sum + (w = kind == run.kind ? work(r) : 0); r = request(++q))
            sum += w;
        // (small units are not cut, where a cut costs more than a step)
        scan[48 + k] = kWhole || run.kind != kOwnKeys ? (int)tree_snap(x, sum, r, TreeCut{steps, ctas}, false) : x;
        if (k == 0) {
            scan[50] = sum;
            scan[51] = q;
        }
    }
    __syncthreads();
    if (works) {
        run.start = scan[48];
        run.end = end < steps ? scan[49] : end;
        run.base = scan[50];
        run.first_b = scan[51];
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
    const SplitRun run =
        split_run<SplitCfg<D, FP8, kTiles, kSets>::kThreads, kTiles, FP8, kSets == 0>(p, reinterpret_cast<int*>(smem));
    TreeCtx c;
    auto two_tiles = [&] {
        tree_setup<D, FP8, 2>(p, smem, c);
        tree_roles<D, FP8, 2, true, FP8 ? kMore : kAll>(p, c, run);
    };
    auto one_tile = [&] {
        tree_setup<D, FP8, 1>(p, smem, c);
        tree_roles<D, FP8, 1, true, FP8 && kTiles == 2 ? kOneTileOnly : kAll>(p, c, run);
    };
    auto own_keys = [&] {
        if constexpr (kSets == 0) {
            one_tile();
        } else {
            few_setup<D, FP8, kSets>(p, smem, c);
            few_roles<D, FP8, kSets>(p, c, run);
        }
    };
    if constexpr (kTiles == 1) {
        run.kind == kOneTile ? one_tile() : own_keys();
    } else if constexpr (FP8 && kSets > 0) {
        if (run.kind == kTwoTiles)
            two_tiles();
        else
            run.kind == kOneTile ? one_tile() : own_keys();
    } else {
        run.kind == kTwoTiles ? two_tiles() : own_keys();
    }
}

}  // namespace

template <int D, bool FP8, int kTiles, int kSets>
cudaError_t launch_split(const TreeParams& q, cudaStream_t stream)
{
    using C = SplitCfg<D, FP8, kTiles, kSets>;
    TreeParams p = q;
    // What steps take, found by timing.  Batch: 64 single tokens of 8 x 4 heads behind 16384
    // shared keys, bf16; groups: 100 of 8 x 8 heads in 8 groups of 3 to 24, e4m3.
    //   step[0], batch: 2 / 2.5 / 3: 53 / 51 / 56 us;  groups: 3 / 3.75 / 4.25: 86 / 77 / 77, with 17
    //   requests each at least: 115 / 107 / 111
    //   step[1], groups: 1.75 / 2.25 / 2.75: 82 / 77 / 83;  with at most 16 requests each, where
    //   that is the only kind of prefix (kTiles 1): 1.25 / 1.75 / 2.25: 76 / 66 / 65
    //   own_cost 1 / 2 / 3: batch 53 / 51 / 53, groups 80 / 77 / 83
    // Other shapes have the same numbers, which are not the best for all.  The batch at D = 64:
    // 38 us, 40 with step[0] 2, 42 with 3.  With 16 heads per kv head (two sets of rows, whose own keys take
    // longer): the batch 43, 38 with step[0] 2; the groups 78, 74 with step[0] 3, 73 with own_cost 3.
    //   own keys by query tiles, step[0], batch: 0.75 / 1.5 / 2 / 3: 102 / 72 / 61 / 62
    if (kSets > 0) {
        p.prefix.own_cost = 2;
        p.prefix.step[0] = FP8 ? 3.75f : 2.5f;
        p.prefix.step[1] = !FP8 ? 1.5f : kTiles == 2 ? 2.25f : 1.75f;
    } else {
        p.prefix.step[0] = FP8 ? 1.5f : 2.f;
        p.prefix.step[1] = 1.f;
    }
    return launch_per_sm<prefix_split_kernel<D, FP8, kTiles, kSets>>(p, C::kThreads, C::kSmemBytes, stream);
}

}  // namespace b2pa
