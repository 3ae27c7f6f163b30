// attn_tree.cu -- attention of drafted token trees: the instantiations of
// attention_tree_kernel (attn_tree.cuh) for trees, and the merge of their
// partial rows.
#include "attn_tree.cuh"

namespace b2pa {

namespace {

// ---------------------------------------------------------------------------
// The merge of a unit that several CTAs shared: with the segments' (m_c, l_c,
// O_c) and m = max m_c, w_c = 2^(m_c - m),
//   out = bmm2 * sum_c w_c O_c / (sum_c w_c l_c + [sinks] 2^(sink log2 e - m)),
// in the order of the keys.  Block (i, y) takes the unit whose first segment is
// CTA i's, if there is one that goes on in the next CTA, and of its query tile
// y / 4 the 32 MMA rows of quadrant y % 4: a lane per row, so that the partial
// rows, four columns of all 128 rows together, are read and were written in
// whole lines.  Each warp takes kCols4 groups of four columns.  Latency alone:
// loads that do not depend on each other are issued together.
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(D * 2) tree_merge_kernel(const __grid_constant__ TreeParams p, int tiles)
{
    constexpr float kLog2e = 1.4426950408889634f;
    constexpr int kCols4 = 4;  // D / 16 warps
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int first = blockIdx.x, qt = (int)blockIdx.y / 4, row = (int)blockIdx.y % 4 * 32 + lane;
    // the segment that opens a unit is the CTA's last; the ones after it are
    // the first of the CTAs that follow, up to the one that reaches the end
    const int4* notes = p.part_seg;
    TreePart x = TreePart::read(notes + (long long)first * 4);
    const TreePart last = TreePart::read(notes + (long long)first * 4 + 2);
    TreePart next = TreePart{};
    if (first + 1 + lane < p.grid)
        next = TreePart::read(notes + (long long)(first + 1 + lane) * 4);
    const int slot = last.all != 0 ? 1 : 0;
    if (slot)
        x = last;
    const int toks = min(p.rows.tile_toks, x.toks - qt * p.rows.tile_toks);
    if (x.all == 0 || x.off != 0 || toks <= 0)
        return;
    int segs = 1;
    for (int c = first + 1;; c += 32) {
        if (c > first + 1)
            next = c + lane < p.grid ? TreePart::read(notes + (long long)(c + lane) * 4) : TreePart{};
        const unsigned m = __ballot_sync(0xffffffffu, next.off + next.tiles >= next.all);  // (none: 0 >= 0)
        if (m != 0) {
            segs += __ffs(m);
            break;
        }
        segs += 32;
    }
    const TreeToken at = tree_token(p.rows, row, toks);
    if (!__any_sync(0xffffffffu, at.valid))
        return;
    // segment c of the unit: slot 0 of CTA first + c, but for its first
    auto part = [&](int c) { return (long long)((first + c) * 2 + (c == 0 ? slot : 0)) * tiles + qt; };
    const int h = x.kvh * p.rows.G + at.head;
    const float sink = p.sinks != nullptr && at.valid ? p.sinks[h] * kLog2e : -INFINITY;
    float m = -INFINITY, den = 0.f;
    float4 a[kCols4];
#pragma unroll
    for (int k = 0; k < kCols4; ++k)
        a[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kBatch = 4;  // segments loaded together
    for (int c0 = 0; c0 < segs; c0 += kBatch) {
        float2 ml[kBatch];
        float4 v[kBatch][kCols4];
#pragma unroll
        for (int c = 0; c < kBatch; ++c) {
            ml[c] = make_float2(-INFINITY, 0.f);
            if (c0 + c < segs && at.valid) {
                const long long q = part(c0 + c);
                ml[c] = p.part_ml[q * kQRows + row];
#pragma unroll
                for (int k = 0; k < kCols4; ++k)
                    v[c][k] = p.part_o[(q * (D / 4) + warp * kCols4 + k) * kQRows + row];
            }
        }
        float top = m;
#pragma unroll
        for (int c = 0; c < kBatch; ++c)
            top = fmaxf(top, ml[c].x);
        const float old = m == top ? 1.f : ex2_approx(m - top);  // (no maximum yet: sums of 0 or NaN)
        m = top;
        den *= old;
#pragma unroll
        for (int k = 0; k < kCols4; ++k)
            a[k] = make_float4(a[k].x * old, a[k].y * old, a[k].z * old, a[k].w * old);
#pragma unroll
        for (int c = 0; c < kBatch; ++c) {
            if (c0 + c >= segs || !at.valid)
                break;
            // (nothing is left out where a weight is 0: a part that is no number, of a
            // maximum below all others' or of none, stays so)
            const float w = ml[c].x == top ? 1.f : ex2_approx(ml[c].x - top);
            den = fmaf(w, ml[c].y, den);
#pragma unroll
            for (int k = 0; k < kCols4; ++k) {
                a[k].x = fmaf(w, v[c][k].x, a[k].x);
                a[k].y = fmaf(w, v[c][k].y, a[k].y);
                a[k].z = fmaf(w, v[c][k].z, a[k].z);
                a[k].w = fmaf(w, v[c][k].w, a[k].w);
            }
        }
    }
    if (!at.valid)
        return;
    if (m != -INFINITY)
        den += ex2_approx(sink - m);
    const float f = den == 0.f ? 0.f : p.bmm2 / den;
    const int tok = x.row0 + qt * p.rows.tile_toks + at.tok;
    uint16_t* to = p.out + (long long)tok * p.out_st_tok + (long long)h * p.out_st_head + warp * kCols4 * 4;
#pragma unroll
    for (int k = 0; k < kCols4; k += 2)
        *reinterpret_cast<uint4*>(to + 4 * k) =
            make_uint4(pack_bf16x2(a[k].x * f, a[k].y * f), pack_bf16x2(a[k].z * f, a[k].w * f),
                       pack_bf16x2(a[k + 1].x * f, a[k + 1].y * f), pack_bf16x2(a[k + 1].z * f, a[k + 1].w * f));
}

template <int D, bool FP8, int kTiles>
cudaError_t launch_tree(const TreeParams& p, cudaStream_t stream)
{
    const cudaError_t e = launch_tree_kernel<D, FP8, kTiles, false>(p, stream);
    if (e != cudaSuccess || p.whole)
        return e;
    return launch_pdl(tree_merge_kernel<D>, dim3(p.grid, 4 * kTiles), D * 2, 0, stream, p, kTiles);
}

}  // namespace

cudaError_t launch_attention_tree(const TreeParams& p, bool fp8, int tiles, cudaStream_t stream)
{
    if (p.D == 128) {
        if (fp8)
            return tiles == 1 ? launch_tree<128, true, 1>(p, stream) : launch_tree<128, true, 2>(p, stream);
        return tiles == 1 ? launch_tree<128, false, 1>(p, stream) : launch_tree<128, false, 2>(p, stream);
    }
    if (p.D == 64 && !fp8)
        return tiles == 1 ? launch_tree<64, false, 1>(p, stream) : launch_tree<64, false, 2>(p, stream);
    return cudaErrorInvalidValue;
}

}  // namespace b2pa
