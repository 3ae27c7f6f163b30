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
#include <algorithm>

#include "attn_split.cuh"

namespace b2pa {

namespace {

// Block (x, b): 32 of request b's rows (kv head, token, head of it), a lane each;
// each warp takes four groups of four columns.  Parts are added in the order of
// the keys.  Latency alone: loads that do not depend on one another are issued
// together.
template <int D>
__global__ void __launch_bounds__(D * 2, 2) prefix_merge_kernel(const __grid_constant__ TreeParams p)
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
    const bool valid = row < all;
    const int per = own.n * G, kvh = valid ? row / per : 0, in = valid ? row - kvh * per : 0;
    const int tok = own.q0 + in / G, h = kvh * G + in % G;
    const long long at = ((long long)kvh * p.T + own.q0) * G + in;
    // (both records, although there may be no prefix: that is known an access later)
    PrefixRow x[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        x[i] = PrefixRow::unpack(p.prefix.part_rec[i][at], at);
    const float sink = p.sinks != nullptr ? p.sinks[h] * kLog2e : -INFINITY;
    bool shared = false;
    if (g >= 0) {
        const TreeReq r = prefix_request(p, g, 1);
        if (!r.ok)
            return;
        shared = r.kv_len > 0;
    }
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
    float4 v[2][kCols4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (valid && (i == kPrefixOwn || shared))
            load(p.prefix.part_o[i], at - x[i].tile_row, x[i], v[i]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (!valid || !(i == kPrefixOwn || shared))
            continue;
        // the rest of the unit: parts of the CTAs behind, looked at kBatch together
        constexpr int kBatch = 2;
        bool more = x[i].cta >= 0 && x[i].cta < p.grid;
        for (int c0 = x[i].cta + 1, first = 1; first || more; c0 += kBatch, first = 0) {
            float2 ml[kBatch];
            float4 z[kBatch][kCols4];
            bool ends[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int c = c0 + k;
                ends[k] = true;
                ml[k] = make_float2(-INFINITY, 0.f);
                if (more && c < p.grid) {
                    const long long rows0 = (long long)(c * 2 + x[i].qt) * kQRows;
                    const float4 y = p.prefix.cut_rec[rows0 + x[i].tile_row];
                    ml[k] = make_float2(y.x, y.y);
                    ends[k] = p.prefix.cut_ends[c] != 0;
                    load(p.prefix.cut_o, rows0, x[i], z[k]);
                }
            }
            if (first)
                merge(x[i].m, x[i].l, v[i]);
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (more) {
                    merge(ml[k].x, ml[k].y, z[k]);
                    more = !ends[k];
                }
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

template <int D, bool FP8>
cudaError_t launch_prefix(TreeParams& p, int tiles, bool few, cudaStream_t stream)
{
    const int G = p.rows.G;
    p.prefix.own_cost = kTreeUnitCost;
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
    const long long rows = (long long)std::min(p.max_q_len, p.T) * p.H;
    if (rows == 0)
        return e;  // (no request may have a token)
    return launch_pdl(prefix_merge_kernel<D>, dim3((unsigned)((rows + 31) / 32), p.B), D * 2, 0, stream, p);
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
