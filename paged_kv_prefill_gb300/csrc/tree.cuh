// tree.cuh -- parameters and geometry of the tree attention kernels
// (attn_tree.cu, and tree_generic_kernel in generic.cu), filled in ops.cu.
//
// Request b brings n = cum_q[b+1] - cum_q[b] drafted nodes, whose own keys are
// the last n of its kv_len keys; c = kv_len - n keys before them are context.
// Node i sees the context keys j >= lo_i and the node keys whose bit is set in
// its mask row.
#pragma once

#include "common.cuh"

namespace b2pa {

// How the 128 MMA rows of a query tile are dealt out.  With G <= 32 query heads
// per kv head, each of the four softmax warps gets whole tokens (box_toks at
// most, in its first box_toks * G lanes), a tile's tokens being split evenly
// over the warps so that a small tree still uses all four.  With more heads
// row = token * G + head.
struct TreeRows {
    int G, box_toks, tile_toks, by_warp;
};

__host__ __device__ inline TreeRows tree_rows(int G)
{
    TreeRows r;
    r.G = G;
    r.by_warp = G <= 32;
    r.box_toks = r.by_warp ? 32 / G : kQRows / G;
    r.tile_toks = r.by_warp ? 4 * r.box_toks : r.box_toks;
    return r;
}

struct TreeParams {  // 128-byte aligned through its CUtensorMap members
    CUtensorMap tm_q;  // 3-D: (D, H, T), box (64, G, box_toks)
    CUtensorMap tm_k;  // 4-D: (D, P, Hkv, pages), box (64 | 128 bytes, min(P,128), 1, 1)
    CUtensorMap tm_v;
    // plain pointers and strides (elements): the generic kernel's, and the slow
    // path for values that are not finite
    const uint16_t* q;
    const void* k;
    const void* v;
    uint16_t* out;
    long long q_st_tok, q_st_head, out_st_tok, out_st_head;
    long long k_st[3], v_st[3];  // page, head, slot
    const int* cum_q;
    const int* seq_lens;
    const int* block_tables;
    long long bt_stride;
    const unsigned* mask;  // [T, words]
    long long mask_stride;
    const int* positions;  // null without a window
    const float* sinks;    // may be null
    float4* part_o;        // [grid * 2][tiles][D / 4][128] unnormalised partial rows, four columns at a time
    float2* part_ml;       // [grid * 2][tiles * 128] running maximum (log2 units) and sum
    int4* part_seg;        // [grid * 2][2]: TreePart of each partial segment
    unsigned* err;
    TreeRows rows;
    int B, T, H, Hkv, D, page_size, max_pages, num_pages, max_q_len, max_kv_len, mask_words, window;
    int grid;              // CTAs of the attention kernel
    int whole;             // no unit is cut (part_* are null)
    float scale_log2;      // bmm1_scale * log2(e)
    float bmm2;
    unsigned long long wait_limit_ns;
    int inject_stall;
};

// What a unit costs beyond its kv tiles, in kv tiles: its Q, the first scores,
// the tree's own tile and the rows' way out.  (bf16 batch 114 us with 0, 105
// with 2, 104.5 with 4, 105 with 6; e4m3 batch 193, 162, 160 and 160; 512 rows per
// kv head 125, 118, 114.6 and 116.)
constexpr int kTreeUnitCost = 4;

// A request as the kernels see it.  Its work is items * Hkv units (a unit is
// a kv head with the nodes of one item) of `tiles` kv tiles each.
struct TreeReq {
    int q0, n, kv_len, ctx, lo, items, n_lo, tiles;
    int unit;  // steps of a unit: its tiles and what it costs beyond them
    bool ok;
    __device__ __forceinline__ long long work(int Hkv) const { return (long long)items * Hkv * unit; }
};

__device__ __forceinline__ TreeReq tree_request(const TreeParams& p, int b, int item_toks)
{
    const RequestView v = load_request(QStarts{p.cum_q, 0}, p.seq_lens, b, p.max_q_len, p.max_kv_len, p.page_size,
                                       p.max_pages, p.T);
    TreeReq r;
    r.q0 = v.q_start;
    r.n = v.q_len;
    r.kv_len = v.kv_len;
    r.ok = v.ok;
    r.ctx = v.kv_len - v.q_len;
    r.lo = p.window < 0 ? 0 : max(0, r.ctx - p.window);  // no row sees an earlier key
    const bool any = v.ok && v.q_len > 0;
    r.items = any ? (v.q_len + item_toks - 1) / item_toks : 0;
    r.n_lo = any ? r.lo / kKvTile : 0;
    r.tiles = any ? (v.kv_len - 1) / kKvTile - r.n_lo + 1 : 0;
    r.unit = r.tiles + kTreeUnitCost;
    return r;
}

// First context key that a node at position pos sees (ctx: none; the window
// does not say which nodes it sees).
__device__ __forceinline__ int tree_row_lo(int pos, int ctx, int kv_len, int window)
{
    return window < 0 ? 0 : min(ctx, max(0, min(max(pos, ctx), kv_len - 1) - window));
}

// The CTAs cut all requests' units, laid end to end, into equal runs: CTA i of
// g takes [start(i), start(i + 1)).  Of a unit, the first kTreeUnitCost steps are
// no tiles: a run that ends there leaves the whole unit to the next.
struct TreeCut {
    long long total;
    int g;
    __device__ __forceinline__ long long start(int i) const { return total * i / g; }
};

__device__ __forceinline__ TreeCut tree_cut(long long total, int grid)
{
    // two steps per CTA at least: fewer partial rows to merge where there is little
    // work (8 nodes, 2048 keys: 16.6 us with one, 14.3 with two, 15.1 with three)
    return TreeCut{total, (int)min((long long)grid, (total + 1) / 2)};
}

// The end x of a run, in a unit of request r, whose units start at base.  Small
// units are not cut, since what a cut costs (another segment, partial rows, their
// merge) is more than the uneven shares: an end inside one moves to the nearer end
// of the unit.  Small: at most 4 kv tiles, or 8 where a run has hardly more than
// one of them; but not a third of them to a run.  (8 nodes x 4 heads, 8 kv
// heads, cut and whole: 8 requests of 512 keys 16.5 and 14.8 us, 24 of 768 28.2 and
// 26.3, 40 of 512 31.7 and 28.7; but 40 of 768 39.3 and 41.8, one of 512 12.8 and 13.8.)
// `whole`: the host knows that all are small (ops.cu); then there is nothing to merge.
constexpr int kTreeWholeTiles = 4;

__device__ __forceinline__ long long tree_snap(long long x, long long base, const TreeReq& r, const TreeCut& cut, bool whole)
{
    const long long all = (long long)r.unit * cut.g;  // (a run: cut.total / cut.g)
    const bool small = r.tiles <= 8 && all <= 3 * cut.total && (r.tiles <= kTreeWholeTiles || 4 * all >= 3 * cut.total);
    if ((!small && !whole) || r.unit <= 0)
        return x;
    const long long u0 = base + (x - base) / r.unit * r.unit;
    return 2 * (x - u0) < r.unit ? u0 : u0 + r.unit;
}

// What the merge needs to know of a segment that is part of a unit: kv tiles
// off .. off + tiles - 1 of the unit's `all`, for the `toks` query rows from
// row0 and the heads of kv head kvh.  all = 0: there is no such segment.
struct TreePart {
    int all, off, tiles, row0, toks, kvh;
    __device__ __forceinline__ void write(int4* at) const
    {
        at[0] = make_int4(all, off, tiles, row0);
        at[1] = make_int4(toks, kvh, 0, 0);
    }
    static __device__ __forceinline__ TreePart read(const int4* at)
    {
        const int4 x = at[0], y = at[1];
        return TreePart{x.x, x.y, x.z, x.w, y.x, y.y};
    }
};

// Which of the `toks` tokens of a query tile, and which head, an MMA row (0 ..
// 127) is; not valid: nobody's.
struct TreeToken {
    int tok, head;
    bool valid;
};

__device__ __forceinline__ TreeToken tree_token(const TreeRows& r, int row, int toks)
{
    TreeToken t;
    if (r.by_warp) {
        const int per = (toks + 3) / 4, lane = row & 31, in = lane / r.G;
        t.tok = (row >> 5) * per + in;
        t.head = lane - in * r.G;
        t.valid = in < per && t.tok < toks;
    } else {
        t.tok = row / r.G;
        t.head = row - t.tok * r.G;
        t.valid = t.tok < toks;
    }
    return t;
}

// tiles: query tiles per item (1 or 2)
cudaError_t launch_attention_tree(const TreeParams& p, bool fp8, int tiles, cudaStream_t stream);
cudaError_t launch_tree_generic(const TreeParams& p, bool fp8, cudaStream_t stream);

}  // namespace b2pa
