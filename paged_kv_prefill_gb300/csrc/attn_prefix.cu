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
// Where a group has more rows than a query tile, prefixes want two tiles that share
// K and V, and the requests' own keys one, on which both softmax groups work: then
// some CTAs run the one kind of kernel and the others the other
// (prefix_split_kernel).
#include <algorithm>

#include "attn_tree.cuh"

namespace b2pa {

namespace {

template <int D, bool FP8>
struct SplitCfg {
    using Two = TreeCfg<D, FP8, 2>;
    using One = TreeCfg<D, FP8, 1>;
    static constexpr int kThreads = Two::kThreads;
    static constexpr int kSmemBytes = Two::kSmemBytes > One::kSmemBytes ? Two::kSmemBytes : One::kSmemBytes;
    static_assert(One::kThreads == kThreads, "the same roles");
};

template <int D, bool FP8>
__global__ void __launch_bounds__(SplitCfg<D, FP8>::kThreads, 1) prefix_split_kernel(const __grid_constant__ TreeParams p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    pdl_wait();
    const TreeRun run = tree_run<SplitCfg<D, FP8>::kThreads, FP8, true, true>(p, 2 * p.rows.tile_toks, p.rows.tile_toks,
                                                                        reinterpret_cast<long long*>(smem));
    TreeCtx c;
    if (run.own) {
        tree_setup<D, FP8, 1>(p, smem, c);
        tree_roles<D, FP8, 1, true>(p, c, run);
    } else {
        tree_setup<D, FP8, 2>(p, smem, c);
        tree_roles<D, FP8, 2, true>(p, c, run);
    }
}

// Block (x, b): 32 of request b's rows (kv head, token, head of it), a lane each;
// each warp takes four groups of four columns.  Parts are added in the order of
// the keys.  Latency alone: loads that do not depend on one another are issued
// together.
template <int D>
__global__ void __launch_bounds__(D * 2) prefix_merge_kernel(const __grid_constant__ TreeParams p)
{
    constexpr float kLog2e = 1.4426950408889634f;
    constexpr int kCols4 = 4;  // D / 16 warps
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.y, G = p.rows.G;
    const TreeReq own = prefix_request(p, p.prefix.groups + b, 1);
    const int g = prefix_group(p, b);
    if (!own.ok)
        return;
    const int row = blockIdx.x * 32 + lane, all = own.n * p.H;
    if (blockIdx.x * 32 >= all)
        return;
    bool shared = false;
    if (g >= 0) {
        const TreeReq r = prefix_request(p, g, 1);
        if (!r.ok)
            return;
        shared = r.kv_len > 0;
    }
    const bool valid = row < all;
    const int per = own.n * G, kvh = valid ? row / per : 0, in = valid ? row - kvh * per : 0;
    const int tok = own.q0 + in / G, h = kvh * G + in % G;
    const long long at = ((long long)kvh * p.T + own.q0) * G + in;
    const float sink = p.sinks != nullptr ? p.sinks[h] * kLog2e : -INFINITY;
    float m = -INFINITY, den = 0.f;
    float4 a[kCols4];
#pragma unroll
    for (int k = 0; k < kCols4; ++k)
        a[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto load = [&](const float4* o, long long rows0, const PrefixRow& x, float4 v[kCols4]) {
#pragma unroll
        for (int k = 0; k < kCols4; ++k)
            v[k] = o[rows0 * (D / 4) + (long long)(warp * kCols4 + k) * x.tile_rows + x.tile_row];
    };
    auto merge = [&](float x_m, float x_l, const float4 v[kCols4]) {
        const float top = fmaxf(m, x_m);
        const float old = m == top ? 1.f : ex2_approx(m - top);
        // (a sum that is no number keeps its weight, whatever its maximum)
        const float w = x_m == -INFINITY && x_l == 0.f ? 0.f : x_m == top ? 1.f : ex2_approx(x_m - top);
        m = top;
        den = fmaf(den, old, w != 0.f ? w * x_l : 0.f);
#pragma unroll
        for (int k = 0; k < kCols4; ++k) {
            const float4 y = w != 0.f ? v[k] : make_float4(0.f, 0.f, 0.f, 0.f);
            a[k] = make_float4(fmaf(a[k].x, old, w * y.x), fmaf(a[k].y, old, w * y.y), fmaf(a[k].z, old, w * y.z),
                               fmaf(a[k].w, old, w * y.w));
        }
    };
    PrefixRow x[2];
    float4 v[2][kCols4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        x[i] = PrefixRow{-INFINITY, 0.f, -1, 0, 0, 0};
        if (valid && (i == kPrefixOwn || shared))
            x[i] = PrefixRow::unpack(p.prefix.part_rec[i][at], at);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (valid && (i == kPrefixOwn || shared))
            load(p.prefix.part_o[i], at - x[i].tile_row, x[i], v[i]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (valid && (i == kPrefixOwn || shared))
            merge(x[i].m, x[i].l, v[i]);
        for (int c = x[i].cta; c >= 0 && c + 1 < p.grid;) {  // (a lane's own)
            const long long rows0 = (long long)(++c * 2 + x[i].qt) * kQRows;
            const float4 y = p.prefix.cut_rec[rows0 + x[i].tile_row];
            const int ends = p.prefix.cut_ends[c];
            float4 z[kCols4];
            load(p.prefix.cut_o, rows0, x[i], z);
            merge(y.x, y.y, z);
            if (ends)
                break;
        }
    }
    if (!valid)
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

template <int D, bool FP8, int kTiles>
cudaError_t launch_prefix(const TreeParams& p, cudaStream_t stream)
{
    using C = SplitCfg<D, FP8>;
    const cudaError_t e = kTiles == 2 && p.max_q_len <= p.rows.tile_toks
                              ? launch_per_sm<prefix_split_kernel<D, FP8>>(p, C::kThreads, C::kSmemBytes, stream)
                              : launch_tree_kernel<D, FP8, kTiles, true>(p, stream);
    if (e != cudaSuccess)
        return e;
    const long long rows = (long long)std::min(p.max_q_len, p.T) * p.H;
    if (rows == 0)
        return e;  // (no request may have a token)
    return launch_pdl(prefix_merge_kernel<D>, dim3((unsigned)((rows + 31) / 32), p.B), D * 2, 0, stream, p);
}

}  // namespace

cudaError_t launch_attention_prefix(const TreeParams& p, bool fp8, int tiles, cudaStream_t stream)
{
    if (p.D == 128) {
        if (fp8)
            return tiles == 1 ? launch_prefix<128, true, 1>(p, stream) : launch_prefix<128, true, 2>(p, stream);
        return tiles == 1 ? launch_prefix<128, false, 1>(p, stream) : launch_prefix<128, false, 2>(p, stream);
    }
    if (p.D == 64 && !fp8)
        return tiles == 1 ? launch_prefix<64, false, 1>(p, stream) : launch_prefix<64, false, 2>(p, stream);
    return cudaErrorInvalidValue;
}

}  // namespace b2pa
