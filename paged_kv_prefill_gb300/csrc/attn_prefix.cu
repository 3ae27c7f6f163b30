// attn_prefix.cu -- attention of requests in groups that share a cached prefix:
// the instantiations of attention_tree_kernel (attn_tree.cuh) with kPrefix, and
// the merge of their partial rows.
//
// For token i of request b in group g, with s = bmm1 <q, K> over the keys of the
// group's prefix and over the request's own keys up to the token's:
//   out = bmm2 (sum_prefix e^{s-m} V + sum_own e^{s-m} V) / (sum_prefix e^{s-m} + sum_own e^{s-m} [+ e^{sink-m}])
//
// A group's prefix is one unit of work per kv head with the rows of all its
// requests, so that its K and V are read once for up to 256 / G tokens, and it
// is work for the tensor cores; each request's own keys are another, bound by
// HBM.  All units' kv tiles, laid end to end, are cut into equal runs, one per
// CTA.  Every row has two parts at least, so that all rows leave unnormalised
// and a second kernel merges them.
//
// Where that is another kind of work, prefixes and the requests' own keys have CTAs
// of their own (attn_split.cuh).
//
// Measured: 64 single tokens of 8 x 4 heads, D = 128, behind 16384 shared keys and 64 to
// 1024 of their own: 51 us, 3.9 TB/s (0.59 of the copy rate); 100 tokens of 8 x 8 heads in 8
// groups over an e4m3 cache: 77 us, 0.53; 16 questions of 16 to 64 tokens behind 32768 keys,
// D = 64: 194 us, 914 TFLOP/s (0.47 of the bf16 rate); 8 samples of one prompt of 2048
// keys: 15.2 us, latency.
#include <algorithm>

#include "attn_split.cuh"

namespace b2pa {

namespace {

// Block (x, y): 32 of all rows (kv head, token, head of it), a lane each, and
// kMergeWarps * kMergeCols4 * 4 columns from y times that on: as many blocks as rows
// take, whatever the bounds on the requests say.  Parts are added in the
// order of the keys.  Latency alone, about four accesses that depend on one another:
// the row's records and the search for its request, lengths, its parts; so nothing
// waits to know whether it is needed (what was not written is read within the
// workspace and left out), a unit's further parts are loaded kBatch together, and a row's
// columns are spread over several SMs (a block of all of them had 1200
// instructions for each of 16 warps).
constexpr int kMergeCols4 = 4, kMergeWarps = 2;

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) prefix_merge_kernel(const __grid_constant__ TreeParams p)
{
    constexpr float kLog2e = 1.4426950408889634f;
    constexpr int kBatch = 4, kCols4 = kMergeCols4;
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
    const unsigned G = p.rows.G, rows = (unsigned)p.T * (unsigned)p.H;
    const unsigned at = min(blockIdx.x * 32 + lane, rows - 1);  // (the last row several times)
    const unsigned kvh = at / (p.T * G), in = at - kvh * (p.T * G);
    const int tok = (int)(in / G), h = (int)(kvh * G + in % G);
    PrefixRow x[2];
    float4 v[2][kCols4];
    auto load = [&](const float4* o, long long rows0, const PrefixRow& x, float4 v[kCols4]) {
#pragma unroll
        for (int k = 0; k < kCols4; ++k)
            v[k] = o[rows0 * (D / 4) + (long long)(warp * kCols4 + k) * x.tile_rows + x.tile_row];
    };
#pragma unroll
    for (int i = 0; i < 2; ++i)
        x[i] = PrefixRow::unpack(p.prefix.part_rec[i][at], at);
    const float sink = p.sinks != nullptr ? p.sinks[h] * kLog2e : -INFINITY;
    const Rising cum(p.cum_q, p.B), groups = prefix_groups(p);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        load(p.prefix.part_o[i], (long long)at - x[i].tile_row, x[i], v[i]);
    TreeReq own;
    const int b = prefix_owner(p, cum, tok, &own), g = prefix_group(p, groups, b);
    const TreeReq group = prefix_request(p, max(g, 0), 1);  // (of no group: not used)
    const bool mine = blockIdx.x * 32 + lane < rows && b >= 0 && !(g >= 0 && !group.ok);
    const bool shared = g >= 0 && group.kv_len > 0;
    float m = -INFINITY, den = 0.f;
    float4 a[kCols4];
#pragma unroll
    for (int k = 0; k < kCols4; ++k)
        a[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto merge = [&](float x_m, float x_l, const float4 v[kCols4]) {
        // (nothing is left out where a weight is 0: a part that is no number, of a maximum
        // below all others' or of none, stays so)
        const float top = fmaxf(m, x_m);
        const float old = m == top ? 1.f : ex2_approx(m - top), w = x_m == top ? 1.f : ex2_approx(x_m - top);
        m = top;
        den = fmaf(den, old, w * x_l);
#pragma unroll
        for (int k = 0; k < kCols4; ++k)
            a[k] = make_float4(fmaf(a[k].x, old, w * v[k].x), fmaf(a[k].y, old, w * v[k].y),
                               fmaf(a[k].z, old, w * v[k].z), fmaf(a[k].w, old, w * v[k].w));
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool some = mine && (i == kPrefixOwn || shared);
        if (some)
            merge(x[i].m, x[i].l, v[i]);
        // the rest of the unit: parts of the CTAs behind
        bool more = some && x[i].cta >= 0 && x[i].cta < p.grid;
        for (int c0 = x[i].cta + 1; __any_sync(0xffffffffu, more); c0 += kBatch) {
            float2 ml[kBatch];
            float4 z[kBatch][kCols4];
            unsigned ends = 0;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int c = more ? min(c0 + k, p.grid - 1) : 0;
                const long long rows0 = (long long)(c * 2 + x[i].qt) * kQRows;
                const float4 y = p.prefix.cut_rec[rows0 + x[i].tile_row];
                ml[k] = make_float2(y.x, y.y);
                ends |= (unsigned)(p.prefix.cut_ends[c] != 0 || c0 + k >= p.grid - 1) << k;
                load(p.prefix.cut_o, rows0, x[i], z[k]);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (more) {
                    merge(ml[k].x, ml[k].y, z[k]);
                    more = !(ends >> k & 1u);
                }
        }
    }
    if (!mine)
        return;
    if (m != -INFINITY)
        den += ex2_approx(sink - m);
    const float f = den == 0.f ? 0.f : p.bmm2 / den;
    uint16_t* to = p.out + (long long)tok * p.out_st_tok + (long long)h * p.out_st_head + warp * kCols4 * 4;
#pragma unroll
    for (int k = 0; k < kCols4; k += 2)
        *reinterpret_cast<uint4*>(to + 4 * k) =
            make_uint4(pack_bf16x2(a[k].x * f, a[k].y * f), pack_bf16x2(a[k].z * f, a[k].w * f),
                       pack_bf16x2(a[k + 1].x * f, a[k + 1].y * f), pack_bf16x2(a[k + 1].z * f, a[k + 1].w * f));
}

template <int D, bool FP8>
cudaError_t launch_prefix(TreeParams& p, int tiles, bool few, cudaStream_t stream)
{
    const int G = p.rows.G;
    const long long rows = (long long)p.T * p.H;
    if (rows > 0x7FFFFFFF)  // (more than 2^40 bytes of workspace)
        return cudaErrorInvalidValue;
    p.prefix.own_cost = kTreeUnitCost;
    // The batch and the groups of attn_split_impl.cuh: 73 and 163 us with all work in one
    // kind of CTA, 62 and 126 with own keys by query tiles on CTAs of their own, 51 and 77 with
    // single tokens' by warps.  A request of more than a query tile is the same work as a
    // prefix, and has nothing from the split.
    cudaError_t e;
    if (few && p.prefix.split)
        e = tiles == 1 ? G <= 8 ? launch_split<D, FP8, 1, 1>(p, stream) : launch_split<D, FP8, 1, 2>(p, stream)
                       : G <= 8 ? launch_split<D, FP8, 2, 1>(p, stream) : launch_split<D, FP8, 2, 2>(p, stream);
    else if (tiles == 2 && p.max_q_len <= p.rows.tile_toks && p.prefix.split)
        e = launch_split<D, FP8, 2, 0>(p, stream);
    else
        e = tiles == 1 ? launch_tree_kernel<D, FP8, 1, true>(p, stream) : launch_tree_kernel<D, FP8, 2, true>(p, stream);
    if (e != cudaSuccess)
        return e;
    const dim3 grid((unsigned)((rows + 31) / 32), D / (4 * kMergeCols4 * kMergeWarps));
    return launch_pdl(prefix_merge_kernel<D>, grid, 32 * kMergeWarps, 0, stream, p);
}

}  // namespace

cudaError_t launch_attention_prefix(const TreeParams& q, bool fp8, int tiles, bool few, cudaStream_t stream)
{
    TreeParams p = q;
    if (p.D == 128)
        return fp8 ? launch_prefix<128, true>(p, tiles, few, stream) : launch_prefix<128, false>(p, tiles, few, stream);
    if (p.D == 64 && !fp8)
        return launch_prefix<64, false>(p, tiles, few, stream);
    return cudaErrorInvalidValue;
}

}  // namespace b2pa
