// tree.cuh -- parameters and geometry of the kernels for a few rows per request
// (attn_tree.cuh, and tree_generic_kernel and prefix_generic_kernel in
// generic.cu), filled in ops.cu: attention of drafted token trees, and of
// requests that share a prefix (kPrefix; see prefix_request).
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

// What the attention of requests with shared prefixes has besides: requests
// cum_groups[g] .. cum_groups[g + 1] - 1 share the prefix of row g of `tables`.
// Rows leave unnormalised, with their maximum and sum: part_*[kPrefixShared] and
// [kPrefixOwn] hold, for each (kv head, token, head of it), the segment that
// begins with the first key of the prefix, and of the request's own keys;
// cut_* what each CTA's first segment continues.
enum { kPrefixShared = 0, kPrefixOwn = 1, kPrefixCut = 2 };
struct PrefixParams {
    const int* tables;
    long long stride;
    const int* lens;
    const int* cum_groups;
    int groups, max_pages, max_len;
    float4* part_o[2];    // [Hkv * T * G] rows, those of a tile together, four columns of all of them at a time
    float4* part_rec[2];  // [Hkv * T * G] PrefixRow
    float4* cut_o;        // [grid * 2][128 rows], the same
    float4* cut_rec;      // [grid * 2][128]
    int* cut_ends;        // [grid]: whether the unit ends there
    // where prefixes and own keys have CTAs of their own: what a step (a kv tile, or
    // one of those that a unit costs beyond them) of a prefix with two query tiles, and
    // with one, takes against one of a request's own; and how many of the latter a unit costs
    float step[2];
    int own_cost;
    bool split;           // all units' steps fit 31 bits
};

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
    PrefixParams prefix;
};

// What a unit of the tree attention's kernel costs beyond its kv tiles, in kv tiles: its Q, the first scores,
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

// (of a shared prefix, whose units are cut between many CTAs, with a first segment
// each: 8 samples 15.1 us with 1, 15.2 with 2, 15.8 with 4; 8 e4m3 groups 83, 77 and 82)
constexpr int kPrefixUnitCost = 2;

// The same of requests that share prefixes.  They are attended as groups + B of
// them: group g's rows, all of its requests' tokens, over the keys of its prefix
// (all context); and each request's rows over its own keys, the last n of which
// are its tokens' (token i sees those up to its own; a single token sees all, so
// that they are all context).
__device__ __forceinline__ TreeReq prefix_request(const TreeParams& p, int v, int item_toks)
{
    const PrefixParams& x = p.prefix;
    TreeReq r;
    if (v < x.groups) {
        const int r0 = x.cum_groups[v], r1 = x.cum_groups[v + 1];
        r.kv_len = x.lens[v];
        r.ok = r0 >= 0 && r0 <= r1 && r1 <= p.B && r.kv_len >= 0 && r.kv_len <= x.max_len &&
               ((long long)r.kv_len + p.page_size - 1) / p.page_size <= x.max_pages;
        r.q0 = r.ok ? p.cum_q[r0] : 0;
        r.n = r.ok ? p.cum_q[r1] - r.q0 : 0;
        r.ok = r.ok && r.n >= 0 && r.q0 >= 0 && r.q0 <= p.T - r.n;
        r.ctx = r.kv_len;
    } else {
        const RequestView w = load_request(QStarts{p.cum_q, 0}, p.seq_lens, v - x.groups, p.max_q_len, p.max_kv_len,
                                           p.page_size, p.max_pages, p.T);
        r.q0 = w.q_start;
        r.n = w.q_len;
        r.kv_len = w.kv_len;
        r.ok = w.ok;
        r.ctx = w.kv_len - (w.q_len > 1 ? w.q_len : 0);
    }
    r.lo = r.n_lo = 0;
    const bool any = r.ok && r.n > 0 && r.kv_len > 0;
    r.items = any ? (r.n + item_toks - 1) / item_toks : 0;
    r.tiles = any ? (r.kv_len - 1) / kKvTile + 1 : 0;
    r.unit = r.tiles + (v < x.groups ? kPrefixUnitCost : x.own_cost);
    return r;
}

__device__ __forceinline__ const int* prefix_pages(const TreeParams& p, int v)
{
    return v < p.prefix.groups ? p.prefix.tables + (long long)v * p.prefix.stride
                               : p.block_tables + (long long)(v - p.prefix.groups) * p.bt_stride;
}

template <bool kPrefix>
__device__ __forceinline__ TreeReq request_of(const TreeParams& p, int v, int item_toks)
{
    return kPrefix ? prefix_request(p, v, item_toks) : tree_request(p, v, item_toks);
}
template <bool kPrefix>
__device__ __forceinline__ int requests_of(const TreeParams& p)
{
    return kPrefix ? p.prefix.groups + p.B : p.B;
}

// Numbers that rise, to be looked through by a whole warp: each lane holds one of 32
// of them, so that a search ends in registers or in the few between two of these.
struct Rising {
    const int* x;
    int n, step, some;
    __device__ __forceinline__ Rising(const int* x_, int n_) : x(x_), n(n_), step(n_ / 32 + 1)
    {
        const int lane = threadIdx.x & 31;
        some = lane * step < n ? x[lane * step] : 0x7FFFFFFF;
    }
    // The last i with x[i] <= value, a lane's own; -1: none.
    __device__ __forceinline__ int last_at_most(int value) const
    {
        int lo = 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            lo += __shfl_sync(0xffffffffu, some, lo + o) <= value && (lo + o) * step < n ? o : 0;
        if (__shfl_sync(0xffffffffu, some, lo) > value || lo * step >= n)
            return -1;
        int hi = min(lo * step + step, n) - 1;
        lo *= step;
        while (lo < hi) {
            const int mid = lo + (hi - lo + 1) / 2;
            if (x[mid] <= value)
                lo = mid;
            else
                hi = mid - 1;
        }
        return lo;
    }
};

// The group of request b, by a whole warp; -1: none.  (Of empty groups that start
// there, the last starts the one that holds b.)
__device__ __forceinline__ Rising prefix_groups(const TreeParams& p) { return Rising(p.prefix.cum_groups, p.prefix.groups + 1); }
__device__ __forceinline__ int prefix_group(const TreeParams& p, const Rising& groups, int b)
{
    const int g = groups.last_at_most(b);
    return g < p.prefix.groups ? g : -1;
}

// The request whose token tok is, by a whole warp; -1: it is nobody's, or a malformed
// request's.  cum: cum_q's first B; *r: that request.
__device__ __forceinline__ int prefix_owner(const TreeParams& p, const Rising& cum, int tok, TreeReq* r)
{
    auto owns = [&](int b) {
        *r = prefix_request(p, p.prefix.groups + b, 1);
        return r->ok && tok >= r->q0 && tok < r->q0 + r->n;
    };
    int b = max(cum.last_at_most(tok), 0);
    bool found = owns(b);
    if (!__all_sync(0xffffffffu, found)) {
        // behind the last request or before the first; else something is malformed, cum_q
        // may fall, and all requests are asked
        const int lane = threadIdx.x & 31;
        int least = 0x7FFFFFFF, most = -0x7FFFFFFF;
        for (int i = lane; i <= p.B; i += 32) {
            least = min(least, p.cum_q[i]);
            most = max(most, p.cum_q[i]);
        }
        least = __reduce_min_sync(0xffffffffu, least);
        most = __reduce_max_sync(0xffffffffu, most);
        if (tok >= least && tok < most)
            for (int i = 0; i < p.B && !found; ++i)
                if (p.cum_q[i] <= tok && tok < p.cum_q[i + 1])
                    found = owns(b = i);
        __syncwarp();
    }
    return found ? b : -1;
}

// A partial row: its maximum (log2 units) and sum; the CTA whose successors
// have the rest of its keys (-1: there is none); how many rows its tile has,
// which of them it is, and which query tile of its CTA that is.
struct PrefixRow {
    float m, l;
    int cta, tile_rows, tile_row, qt;
    __device__ __forceinline__ float4 pack() const
    {
        return make_float4(m, l, __int_as_float(cta), __int_as_float(tile_rows | tile_row << 8 | qt << 16));
    }
    // Row `at` of its plane.  (After a wait that gave up, rows were not written:
    // whatever they hold stays within the workspace.)
    static __device__ __forceinline__ PrefixRow unpack(float4 x, long long at)
    {
        const int w = __float_as_int(x.w), rows = min(w & 255, kQRows);
        return PrefixRow{x.x, x.y, __float_as_int(x.z), rows, (int)min((long long)min(w >> 8 & 255, kQRows - 1), at),
                         w >> 16 & 1};
    }
};

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

template <typename Int>  // a 32-bit one where the caller's numbers fit it
__device__ __forceinline__ Int tree_snap(Int x, Int base, const TreeReq& r, const TreeCut& cut, bool whole)
{
    const long long all = (long long)r.unit * cut.g;  // (a run: cut.total / cut.g)
    const bool small = r.tiles <= 8 && all <= 3 * cut.total && (r.tiles <= kTreeWholeTiles || 4 * all >= 3 * cut.total);
    if ((!small && !whole) || r.unit <= 0)
        return x;
    const Int u0 = base + (x - base) / r.unit * r.unit;
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
// tiles: query tiles per item of a prefix; few: the requests' own keys with
// attn_few.cuh
cudaError_t launch_attention_prefix(const TreeParams& p, bool fp8, int tiles, bool few, cudaStream_t stream);
cudaError_t launch_prefix_generic(const TreeParams& p, bool fp8, cudaStream_t stream);
cudaError_t launch_tree_generic(const TreeParams& p, bool fp8, cudaStream_t stream);

}  // namespace b2pa
